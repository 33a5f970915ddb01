"""The barriers of the 256-wide attention kernel, every interleaving of its
warps: no wait may be left behind by two phases of its barrier (a parity then
reads as if nothing had happened, and the wait hangs until its limit).

Each role is the list of its waits and arrivals, in program order, for units of
given numbers of blocks.  The softmax warps are one role (all of them wait and
arrive alike), and so is the pair of a product and its commit."""
import pytest

RING = 4            # stages of the ring that K goes through


def _roles(units, seen):
    """Waits (barrier, phase) and arrivals (barrier,) of every role; `seen`:
    the score warps say that they have seen a unit's q, and the next q is
    announced after that only."""
    softmax, weights, keys = [], [], []
    scores = [[], []]
    bring = lambda u: ([("q_empty", u - 1)] if seen and u else []) + [("q_full",)]
    softmax += bring(0)
    c = 0
    for u, n in enumerate(units):
        for me in (0, 1):
            scores[me].append(("q_full", u))
            if seen:
                scores[me].append(("q_empty",))
        for _ in range(n):
            slot, use, st, turn = c % 2, c // 2, c % RING, c // RING
            keys += ([(f"k_empty{st}", turn - 1)] if turn else []) + [(f"k_full{st}",)]
            for me in (0, 1):
                mine = slot == me
                if mine and c >= 2:
                    scores[me].append((f"pv_done{slot}", use - 1))
                scores[me].append((f"k_full{st}", turn))
                if mine:
                    scores[me].append((f"s_full{slot}",))
                scores[me].append((f"k_empty{st}",))
            softmax += [(f"s_full{slot}", use), (f"p_full{slot}",)]
            weights += [(f"p_full{slot}", use), (f"pv_done{slot}",)]
            c += 1
        if u + 1 < len(units):
            softmax += bring(u + 1)
        softmax.append((f"pv_done{(c - 1) % 2}", (c - 1) // 2))
    return [softmax, weights, keys, *scores]


def _fault(units, seen):
    """A wait that two phases can pass by, or a standstill; None if there is neither."""
    roles = _roles(units, seen)
    names = sorted({op[0] for r in roles for op in r})
    index = {n: i for i, n in enumerate(names)}
    need = {n: 2 if n.startswith(("k_empty", "q_empty")) else 1 for n in names}
    start = (tuple([0] * len(roles)), tuple([(0, 0)] * len(names)))      # (phases done, arrivals in this one)
    todo, known = [start], {start}
    while todo:
        at, bars = todo.pop()
        moved = False
        for r, ops in enumerate(roles):
            if at[r] == len(ops):
                continue
            op = ops[at[r]]
            i = index[op[0]]
            done, n = bars[i]
            new = bars
            if len(op) == 2:
                if done > op[1] + 1:
                    return f"{op[0]}: phase {op[1]} passed by"
                if done <= op[1]:
                    continue
            else:
                n += 1
                new = list(bars)
                new[i] = (done + 1, 0) if n == need[op[0]] else (done, n)
                new = tuple(new)
            moved = True
            state = (at[:r] + (at[r] + 1,) + at[r + 1:], new)
            if state not in known:
                known.add(state)
                todo.append(state)
        if not moved and any(a < len(o) for a, o in zip(at, roles)):
            return "standstill"
    return None


@pytest.mark.parametrize("units", [[1, 1, 1, 1, 1], [1, 2, 1, 1], [3, 1, 1, 2], [2, 2, 2], [5, 1, 4], [1, 7]])
def test_no_wait_is_passed_by(units):
    assert _fault(units, seen=True) is None


def test_q_announced_without_the_score_warps_can_pass_by():
    """The model sees the fault: with units of one block, whose scores only one of the two warps computes."""
    assert _fault([1, 1, 1], seen=False).startswith("q_full: phase")
    assert _fault([2, 2, 2], seen=False) is None
