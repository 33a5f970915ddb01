"""The barriers of the adapters' output kernel over a run of several tiles, with the rings that are
launched: h of a tile after that of another, tiles that only copy y between them, and the ends of
the rings.  (test_adapter_protocol.py has the blocks of one tile, on smaller rings, and the notation.)"""
import pytest

import test_adapter_protocol as one_tile

# pieces of y to a column block; places for pieces and for blocks of B: fp16 and fp32 up to rank 64, then above
RINGS = [(2, 8, 4), (4, 8, 4), (2, 6, 2), (4, 4, 3)]


def _run(tiles, pieces, places, b_stages):
    """`tiles`: column blocks of each, negative for tiles that copy y."""
    half = pieces // 2
    bring_b, bring_y, issue, out = [], [], [], [[], []]
    u = c = h = 0                                          # blocks with a product, pieces, tiles with an adapter
    for blocks in tiles:
        copies, blocks = blocks < 0, abs(blocks)
        if not copies:
            bring_b += ([("h_empty", h - 1)] if h else []) + [("h_full", "load")]
            issue.append(("h_full", h))
        for b in range(blocks):
            if not copies:
                st, turn, acc, use = u % b_stages, u // b_stages, u % one_tile.ACCS, u // one_tile.ACCS
                bring_b += ([(f"b_empty{st}", turn - 1)] if turn else []) + [(f"b_full{st}", "load")]
                issue += ([(f"t_empty{acc}", use - 1)] if use else []) + [(f"b_full{st}", turn), (f"b_empty{st}",)]
                issue += [("h_empty",)] if b + 1 == blocks else []
                issue.append((f"t_full{acc}",))
            for p in range(pieces):
                at, turn = (c + p) % places, (c + p) // places
                bring_y += ([(f"y_empty{at}", turn - 1)] if turn else []) + [(f"y_full{at}", "load")]
            for side in (0, 1):
                if not copies:
                    out[side].append((f"t_full{acc}", use))
                for go in range(half):
                    i = c + side * half + go
                    if not copies and go + 1 == half:
                        out[side].append((f"t_empty{acc}",))
                    out[side] += [(f"y_full{i % places}", i // places), (f"y_empty{i % places}",)]
            c += pieces
            u += not copies
        h += not copies
    return [bring_b, bring_y, issue, *out]


def _fault(monkeypatch, tiles, pieces, places, b_stages):
    monkeypatch.setattr(one_tile, "_roles", lambda *_: _run(tiles, pieces, places, b_stages))
    return one_tile._fault(0, 0, 0)


@pytest.mark.parametrize("tiles", [(1, -1, 1), (-1, 2), (3,)])
@pytest.mark.parametrize("pieces,places,b_stages", RINGS)
def test_runs_of_tiles(monkeypatch, tiles, pieces, places, b_stages):
    assert _fault(monkeypatch, tiles, pieces, places, b_stages) is None


@pytest.mark.parametrize("tiles", [(1, 1, 1), (2, -1, 1), (2, 3)])
@pytest.mark.parametrize("pieces,places,b_stages", RINGS[2:])
def test_rings_that_come_round(monkeypatch, tiles, pieces, places, b_stages):
    """More blocks than either ring has places (the larger rings come round too: five blocks in
    fp16 and four in fp32 have no fault either, a minute each and therefore not here)."""
    assert _fault(monkeypatch, tiles, pieces, places, b_stages) is None


def test_places_that_change_hands_are_seen(monkeypatch):
    """fp32 pieces in six places, with a copying tile between two others too."""
    assert _fault(monkeypatch, (4,), 4, 6, 2).endswith("early")
    assert _fault(monkeypatch, (2, -2, 1), 4, 6, 2).endswith("early")


@pytest.mark.parametrize("stages", range(1, 9))
def test_a_kernel_that_gives_up_waits_for_its_copies(stages):
    """The waits of its last uses of a ring (use u: place u % stages, parity of phase u / stages): each blocks
    until that use's copy has come and passes then, whatever has come of the others."""
    for used in range(0, 3 * stages + 2):
        last = range(max(0, used - stages), used)
        assert len({u % stages for u in last}) == len(last)          # at most one copy on its way to each place
        for come in (False, True):
            for u in last:
                phase = u // stages + come                           # phases done at the place
                passes = (phase - 1) % 2 == u // stages % 2          # of a wait on a parity
                assert passes == come
        for u in range(last.start):                                  # earlier copies had come before the place was used again
            assert any(v % stages == u % stages and v > u for v in last)
