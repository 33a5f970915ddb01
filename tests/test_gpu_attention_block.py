"""The attention half of a decoder layer (examples/attention_block.py): EXL3
linears, append, attention and output linear together, a prompt in chunks and
decode steps from a graph, against plain attention in fp64.

Bound: the attention outputs differ by at most 2^-11 (rounding) + 2^-11 (fp16
weights) + the rounding of q and k in the cache (2^-11 each, through the
scores: a relative change of the weights of 2^-10 |s| with |s| of a few units),
a relative error of a few 2^-10 in norm; both sides then go through the same
output linear, whose own tolerance is 1e-3.  5e-3 holds the sum.
"""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [dict(hidden=512, heads_q=4, heads_kv=2, head_dim=128, prompt=300, chunk=128, steps=5),
                                   dict(hidden=512, heads_q=8, heads_kv=2, head_dim=64, prompt=1, chunk=1, steps=40),
                                   dict(hidden=1024, heads_q=8, heads_kv=1, head_dim=256, prompt=700, chunk=700, steps=3)])
def test_block(shape):
    import attention_block
    rel, _, _ = attention_block.run(**shape)
    assert rel <= 5e-3
