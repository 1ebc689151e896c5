"""Model of the own-keys kernel's ring (csrc/attn_prefix_kernel.cuh: attn_prefix_own_kernel), on the CPU.

One warp fills and reads a ring of steps of its own: `issue` asks for a step's K and V, and for the
piece's Q with the piece's first step, where there is a stage (and a place for Q) free; the copies land
in any order at any later time, and a step's barrier completes when all of them have.  Replayed under
many random timings: what is read is what was asked for, no copy goes where something unread
lies, no barrier gets two phases ahead of the wait, and nothing is in flight at the end, after an abort either.
Like the kernel's own documentation, the model states it; when the kernel changes, it changes with it.
"""
import random

import pytest


class Wrong(Exception):
    pass


def run(pieces, stages, seed, q_slots=2, abort_at=None, keep_q=True):
    """One warp over pieces (each so many steps).  None, or what went wrong."""
    rng = random.Random(seed)
    walk = [(p, s, s == 0, s == n - 1) for p, n in enumerate(pieces) for s in range(n)]
    stage = [{"K": None, "V": None} for _ in range(stages)]
    steps = [None] * stages
    done = [0] * stages           # completed phases of a stage's barrier
    missing = [0] * stages        # copies that its current phase still waits for
    q_place, q_unread = [None] * q_slots, [False] * q_slots
    flying = []                   # (stage, what, where, value)
    filled = used = q_filled = q_used = 0

    def land(i):
        st, what, where, value = flying.pop(i)
        if what == "Q":
            if q_unread[where]:
                raise Wrong("Q lands on one that was not read")
            q_place[where], q_unread[where] = value, True
        else:
            stage[st][what] = value
        missing[st] -= 1
        if missing[st] == 0:
            done[st] += 1

    def issue():
        nonlocal filled, q_filled
        if filled == len(walk) or filled - used == stages:
            return False
        p, s, first, _ = walk[filled]
        if first and keep_q and q_filled - q_used == q_slots:
            return False
        st = filled % stages
        if missing[st]:
            raise Wrong("a stage is filled while its copies are in flight")
        steps[st] = walk[filled]
        flying.extend([(st, "K", None, (p, s)), (st, "V", None, (p, s))])
        missing[st] = 2
        if first:
            flying.append((st, "Q", q_filled % q_slots, p))
            missing[st] = 3
            q_filled += 1
        filled += 1
        return True

    def wait(st, phase):
        while done[st] <= phase:
            if not missing[st]:
                raise Wrong("a wait for nothing")
            land(rng.randrange(len(flying)))
        if done[st] > phase + 1:
            raise Wrong("a barrier two phases ahead")

    try:
        while issue():
            pass
        q = None
        while used < filled:
            st = used % stages
            for _ in range(rng.randrange(3)):  # copies land while the warp works
                if flying:
                    land(rng.randrange(len(flying)))
            if used == abort_at:
                break
            wait(st, used // stages)
            p, s, first, last = steps[st]
            if (p, s) != walk[used][:2] or stage[st] != {"K": (p, s), "V": (p, s)}:
                raise Wrong(f"step {walk[used]}: read {steps[st]}, {stage[st]}")
            if first:
                at = q_used % q_slots
                q, q_unread[at] = q_place[at], False
                q_used += 1
            if q != p:
                raise Wrong(f"piece {p} with the queries of {q}")
            used += 1
            while issue():
                pass
        for u in range(used, filled):  # after an abort
            wait(u % stages, u // stages)
        if flying or (abort_at is None and used != len(walk)):
            raise Wrong("left over")
    except Wrong as e:
        return str(e)
    return None


PIECES = [[1], [5], [1] * 9, [1, 7, 2, 1, 1, 3], [2] * 6, [9, 1, 1, 1, 9], []]


@pytest.mark.parametrize("stages", [2, 4])
@pytest.mark.parametrize("pieces", PIECES + [[random.Random(k + i).randint(1, 4) for i in range(10)] for k in range(6)])
def test_ring(pieces, stages):
    for seed in range(40):
        assert run(pieces, stages, seed) is None
        assert run(pieces, stages, seed, abort_at=seed % max(1, sum(pieces))) is None


def test_checker_finds_queries_that_are_written_over():
    """Without the rule on Q's places, short pieces ask for a third piece's Q before the first was read."""
    found = [run([1] * 9, 4, seed, keep_q=False) for seed in range(40)]
    assert any(f and f.startswith("Q lands") for f in found)
