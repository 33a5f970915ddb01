"""exl3_paged_attention where it can go wrong: units of one block, extreme
scores, one key that outweighs a long history, batches whose sequences differ
most.  Helpers and bounds are those of tests/test_gpu_attention.py and
tests/attention_ref.py, unless a test derives a closer bound of its own."""
import pytest

from test_gpu_attention import _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,rows", [(16, 2, 3), (8, 8, 20), (128, 1, 1)])
@pytest.mark.parametrize("B", [1, 30, 160])
def test_units_of_one_block(Hq, Hkv, rows, B):
    """256-wide heads on the tensor cores: every unit has one block of 64 keys, or
    (every fifth sequence) two, so that the two score warps take turns."""
    old = [(i * 13) % (60 - rows) + (64 if i % 5 == 4 else 0) for i in range(B)]
    _run([rows] * B, old, Hq, Hkv, 256)


@pytest.mark.parametrize("rows", [40, 17])
def test_short_units_among_long_ones(rows):
    """256-wide heads: units of one block between units that are cut."""
    old = [0, 9000, 1, 5, 20, 3000, 0, 0, 0, 15, 64, 2, 7000]
    _run([rows] * len(old), old, 8, 4, 256, page=32)
