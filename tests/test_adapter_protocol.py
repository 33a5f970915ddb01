"""The barriers of the adapters' output kernel, every interleaving of its roles and
of its copies' arrivals: no wait may pass before its phase is done, and none may be
left behind by two phases (a parity does not tell these apart).

Each role is the list of its operations in program order: waits (barrier, phase),
arrivals (barrier,) and started copies (barrier, "load"), which arrive at any later
time.  The four warps of a half of the columns act alike and are one role."""
import pytest

ACCS = 2            # accumulators


def _roles(blocks, pieces, places, b_stages):
    """`blocks` column blocks of one tile, `pieces` copies of y each in a ring of `places`."""
    half = pieces // 2
    bring_b, bring_y, issue, out = [], [], [], [[], []]
    for u in range(blocks):
        st, turn = u % b_stages, u // b_stages
        bring_b += ([(f"b_empty{st}", turn - 1)] if turn else []) + [(f"b_full{st}", "load")]
        acc, use = u % ACCS, u // ACCS
        issue += ([(f"t_empty{acc}", use - 1)] if use else []) + [(f"b_full{st}", turn), (f"b_empty{st}",),
                                                                  (f"t_full{acc}",)]
        for p in range(pieces):
            c = u * pieces + p
            place, turn_y = c % places, c // places
            bring_y += ([(f"y_empty{place}", turn_y - 1)] if turn_y else []) + [(f"y_full{place}", "load")]
        for h in (0, 1):
            out[h].append((f"t_full{acc}", use))
            for go in range(half):
                c = u * pieces + h * half + go
                if go + 1 == half:
                    out[h].append((f"t_empty{acc}",))
                out[h] += [(f"y_full{c % places}", c // places), (f"y_empty{c % places}",)]
    return [bring_b, bring_y, issue, *out]


def _fault(blocks, pieces, places, b_stages=2):
    """A wait that passes early or that two phases pass by, or a standstill; None if there is none."""
    roles = _roles(blocks, pieces, places, b_stages)
    names = sorted({op[0] for r in roles for op in r})
    index = {n: i for i, n in enumerate(names)}
    need = [2 if n.startswith("t_empty") else 1 for n in names]
    zero = tuple([0] * len(names))
    start = (tuple([0] * len(roles)), zero, zero, zero)      # (phases done, arrivals in this one, copies on their way)
    todo, known = [start], {start}

    def arrive(done, n, i):
        done, n = list(done), list(n)
        n[i] += 1
        if n[i] == need[i]:
            done[i], n[i] = done[i] + 1, 0
        return tuple(done), tuple(n)

    while todo:
        at, done, n, way = todo.pop()
        after = []
        for i, w in enumerate(way):
            if w:
                after.append((at, *arrive(done, n, i), way[:i] + (w - 1,) + way[i + 1:]))
        for r, ops in enumerate(roles):
            if at[r] == len(ops):
                continue
            op = ops[at[r]]
            i = index[op[0]]
            d2, n2, way2 = done, n, way
            if len(op) == 1:
                d2, n2 = arrive(done, n, i)
            elif op[1] == "load":
                way2 = way[:i] + (way[i] + 1,) + way[i + 1:]
            else:
                if done[i] > op[1] + 1:
                    return f"{op[0]}: phase {op[1]} passed by"
                if done[i] < op[1]:
                    return f"{op[0]}: phase {op[1]} early"
                if done[i] == op[1]:
                    continue
            after.append((at[:r] + (at[r] + 1,) + at[r + 1:], d2, n2, way2))
        if not after and any(a < len(o) for a, o in zip(at, roles)):
            return "standstill"
        for s in after:
            if s not in known:
                known.add(s)
                todo.append(s)
    return None


@pytest.mark.parametrize("b_stages", [1, 2])
@pytest.mark.parametrize("pieces,places,blocks", [(2, 4, 5), (2, 6, 4), (4, 4, 4)])
def test_every_wait_sees_its_own_phase(pieces, places, blocks, b_stages):
    """fp16 (two pieces to a block) and fp32 (four), rings that are whole blocks."""
    assert _fault(blocks, pieces, places, b_stages) is None


def test_places_that_change_hands_can_be_passed_early():
    """The model sees the fault: a place that serves the two halves of the columns in turn."""
    assert _fault(4, 4, 6).endswith("early")
