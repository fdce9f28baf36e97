"""A model of the MXFP4 decoding step's ring, searched exhaustively: two groups of
warps multiply alternate stages, and both wait for every stage by parity.  (A
barrier with `phases` completed phases lets a wait for round r pass when the
parity of `phases` differs from r's, whatever the number of rounds between.)"""

import pytest


def search(slots, stages, both_give_back):
    """Every order of the producer's and the groups' steps; the states in which
    some are left and none can step, and the passes that saw a wrong stage."""
    # filled, full phases, arrivals and phases of empty, each group's (stage, working)
    start = (0, (0,) * slots, (0,) * slots, (0,) * slots, ((0, False), (0, False)))
    need = 2 if both_give_back else 1
    seen, todo, stuck, wrong = {start}, [start], [], []

    def put(t, i, v):
        return t[:i] + (v,) + t[i + 1:]

    while todo:
        state = todo.pop()
        filled, full, arrived, empty, groups = state
        nexts = []
        if filled < stages:
            s, r = filled % slots, filled // slots
            if empty[s] % 2 != (r % 2) ^ 1:
                nexts.append((filled + 1, put(full, s, full[s] + 1), arrived, empty, groups))
        for g, (n, working) in enumerate(groups):
            if n == stages:
                continue
            s, r = n % slots, n // slots

            def give_back():
                if arrived[s] + 1 == need:
                    return put(arrived, s, 0), put(empty, s, empty[s] + 1)
                return put(arrived, s, arrived[s] + 1), empty

            if working:
                nexts.append((filled, full, *give_back(), put(groups, g, (n + 1, False))))
            elif full[s] % 2 != r % 2:
                if full[s] != r + 1:
                    wrong.append(state)
                if n % 2 == g:
                    nexts.append((filled, full, arrived, empty, put(groups, g, (n, True))))
                else:
                    rest = give_back() if both_give_back else (arrived, empty)
                    nexts.append((filled, full, *rest, put(groups, g, (n + 1, False))))
        if not nexts and (filled < stages or any(n < stages for n, _ in groups)):
            stuck.append(state)
        for t in nexts:
            if t not in seen:
                seen.add(t)
                todo.append(t)
    return stuck, wrong


@pytest.mark.parametrize("slots", [2, 3, 5, 6])
def test_both_groups_give_a_stage_back(slots):
    assert search(slots, 4 * slots + 1, True) == ([], [])


@pytest.mark.parametrize("slots", [2, 3, 5, 6])
def test_one_group_alone_would_not_do(slots):
    stuck, _ = search(slots, 4 * slots + 1, False)
    assert stuck
