"""Models of the barrier protocols of the packed kernels' CTAs, on the CPU: attn_packed_kernel.cuh and
attn_packed_bwd_kernel.cuh, replayed under many random interleavings with the kernels' arrival counts (a
warpgroup or warp that always arrives together counts once) and issue order.

Copies land and tensor-core work completes late, at random, the latter in issue order.  Checked: no deadlock; a wait passes
exactly when the phase that it means has completed (a parity cannot tell a phase from the next but one: a wait that
the hardware would let through early, or would miss, fails here); and every buffer (K/V stages, query slots, scores, output
accumulators, row weights, statistics) holds what its reader expects when it is read.  The models state
what the kernels do; when these change, they change with them.  Planted mistakes are caught.
"""
import random

import pytest


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        assert self.pending > 0, "more arrivals than a phase has"
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.phase = self.count, self.phase + 1

    def passes(self, k):
        """A parity wait for the completion of phase k, as the hardware answers it."""
        through = (self.phase ^ k) & 1 == 1
        assert not through or self.phase == k + 1, "let through by an older phase"
        assert through or self.phase <= k, "phase missed"
        return through


class Machine:
    """Runs generators that yield conditions; beside them a queue of copies (any order) and one of MMAs (in order)."""

    def __init__(self, rng):
        self.rng, self.copies, self.mma = rng, [], []

    def run(self, roles):
        waiting = {name: (gen, None) for name, gen in roles.items()}
        while waiting or self.copies or self.mma:
            ready = [n for n, (g, c) in waiting.items() if c is None or c()]
            moves = ready + [self.copies] * bool(self.copies) + [self.mma] * bool(self.mma)
            assert moves, f"deadlock: {sorted(waiting)}"
            m = self.rng.choice(moves)
            if m is self.copies:
                self.copies.pop(self.rng.randrange(len(self.copies)))()
            elif m is self.mma:
                self.mma.pop(0)()
            else:
                gen, _ = waiting.pop(m)
                try:
                    waiting[m] = (gen, next(gen))
                except StopIteration:
                    pass


# ------------------------------------------------------------------ forward
RING = 8


def forward(rng, items, stages, mistake=None):
    """items: (two query tiles, K/V tiles, tiles of the first query tile)."""
    mc = Machine(rng)
    B = {"kvf": [Bar(1) for _ in range(stages)], "kve": [Bar(1) for _ in range(stages)]}
    for n in ("qf", "qe", "sf", "ph", "pf", "of", "oe", "wf", "we"):
        B[n] = [Bar(1), Bar(1)]
    B["x"] = Bar(1)
    B["if"], B["ie"] = [Bar(1) for _ in range(RING)], [Bar(6) for _ in range(RING)]  # producer, MMA, Q, two softmax groups, epilogue
    ring, kv, q = [None] * RING, [None] * stages, [None, None]
    S, P, O, W = [None, None], [None, None], [[], []], {}
    done = {}
    seq = list(items) + [None]

    def take(n):
        yield lambda: B["if"][n % RING].passes(n // RING)
        assert ring[n % RING] == n

    def scheduler():
        for n, it in enumerate(seq):
            if n >= RING:
                yield lambda n=n: B["ie"][n % RING].passes(n // RING - 1)
            ring[n % RING] = n
            B["if"][n % RING].arrive()

    def producer():
        fill = 0
        for n, it in enumerate(seq):
            yield from take(n)
            B["ie"][n % RING].arrive()
            for j in range(it[1] if it else 0):
                for what in "KV":
                    s = fill % stages
                    yield lambda s=s, f=fill: B["kve"][s].passes(f // stages - 1)

                    def land(s=s, tag=(n, j, what)):
                        kv[s] = tag
                        B["kvf"][s].arrive()

                    mc.copies.append(land)
                    fill += 1

    def loader():
        pos = 0
        for n, it in enumerate(seq):
            yield from take(n)
            B["ie"][n % RING].arrive()
            for k in range((2 if it[0] else 1) if it and it[1] else 0):
                yield lambda p=pos: B["qe"][p & 1].passes(p // 2 - 1)

                def land(s=pos & 1, tag=(n, k)):
                    q[s] = tag
                    B["qf"][s].arrive()

                mc.copies.append(land)
                pos += 1

    def mma():
        fill, pos, par = 0, 0, 0  # K/V fills and query tiles before the item, chain of its first step
        p_use, o_use = [0, 0], [0, 0]
        due = []

        def score(c, n, k, j, kf, slot):
            def op():
                assert kv[kf % stages] == (n, j, "K") and q[slot] == (n, k)
                assert P[c] is None, "scores over a P that is still to be read"
                S[c] = (n, j)
                B["sf"][c].arrive()

            mc.mma.append(op)

        def commit(bar):
            mc.mma.append(bar.arrive)

        def output(c, n, j, vf, first, last, last_v):
            yield lambda: B["kvf"][vf % stages].phase > vf // stages or B["kvf"][vf % stages].passes(vf // stages)
            yield lambda u=p_use[c]: B["ph"][c].passes(u)
            if first:
                yield lambda u=o_use[c]: B["oe"][c].passes(u - 1)
                o_use[c] += 1
            yield lambda u=p_use[c]: B["pf"][c].passes(u)
            p_use[c] += 1

            def op():
                assert P[c] == (n, j) and kv[vf % stages] == (n, j, "V")
                if first:
                    assert not O[c], "O not read yet"
                O[c].append((n, j))
                P[c] = None

            mc.mma.append(op)
            if last_v:
                commit(B["kve"][vf % stages])
            if last:
                commit(B["of"][c])

        def run_due():
            if due:
                yield from output(*due.pop())

        for n, it in enumerate(seq):
            if due and B["if"][n % RING].phase <= n // RING:
                yield from run_due()
            yield from take(n)
            B["ie"][n % RING].arrive()
            if not it or it[1] == 0:
                continue
            two, nt, n0 = it
            if two:
                q0, q1 = pos & 1, (pos & 1) ^ 1
                if due and (due[0][0] == 0 or rng.random() < 0.5):
                    yield from run_due()
                for j in range(nt):
                    kf = fill + 2 * j
                    yield lambda kf=kf: B["kvf"][kf % stages].passes(kf // stages)
                    if j == 0:
                        yield lambda: B["qf"][q0].passes(pos // 2)
                        yield lambda: B["qf"][q1].passes((pos + 1) // 2)
                    if j < n0:
                        score(0, n, 0, j, kf, q0)
                        if j == n0 - 1:
                            commit(B["qe"][q0])
                    if j == 0:
                        yield from run_due()
                    else:
                        yield from output(1, n, j - 1, kf - 1, j == 1, False, True)
                    score(1, n, 1, j, kf, q1)
                    commit(B["kve"][kf % stages])
                    if j == nt - 1:
                        commit(B["qe"][q1])
                    if j == n0:
                        commit(B["of"][0])
                    if j < n0:
                        yield from output(0, n, j, kf + 1, j == 0, j == n0 - 1 and n0 == nt, False)
                due.append((1, n, nt - 1, fill + 2 * nt - 1, nt == 1, True, True))
                pos, par = pos + 2, 0
            else:
                for j in range(nt):
                    c, kf = (par + j) & 1, fill + 2 * j
                    if due and rng.random() < 0.5:
                        yield from run_due()
                    yield lambda kf=kf: B["kvf"][kf % stages].passes(kf // stages)
                    if j == 0:
                        yield lambda: B["qf"][pos & 1].passes(pos // 2)
                    score(c, n, 0, j, kf, pos & 1)
                    commit(B["kve"][kf % stages])
                    if j == nt - 1:
                        commit(B["qe"][pos & 1])
                    yield from run_due()
                    due.append((c, n, j, kf + 1, j < 2, j + 2 >= nt, True))
                pos, par = pos + 1, (par + nt) & 1
            fill += 2 * nt
        yield from run_due()

    def softmax(t):
        s_use, x_use, w_use, ring_fill, par = 0, 0, [0, 0], 0, 0
        for n, it in enumerate(seq):
            yield from take(n)
            if not it:
                B["ie"][n % RING].arrive()
                return
            two, nt, n0 = it
            both = two or nt >= 2
            mine = 0 if two else t ^ par
            if nt and (both or mine == 0):
                for j in range(mine, (n0 if t == 0 else nt) if two else nt, 1 if two else 2):
                    yield lambda u=s_use: B["sf"][t].passes(u)
                    s_use += 1
                    assert S[t] == (n, j)
                    if j == nt - 1 and (not two or t == (0 if j < n0 else 1)):  # zeroes what lies behind the last key
                        vf = ring_fill + 2 * j + 1
                        yield lambda vf=vf: B["kvf"][vf % stages].passes(vf // stages)
                        assert kv[vf % stages] == (n, j, "V")
                    P[t] = (n, j)
                    B["ph"][t].arrive()
                    yield None
                    B["pf"][t].arrive()
                merge = both and not two
                yield lambda: B["we"][t].passes(w_use[t] - 1)
                if merge and t == 1:
                    yield lambda: B["we"][0].passes(w_use[0] - 1)
                    W["pair"] = ("stats", n)
                    (B["wf"][1] if mistake == "shared exchange" else B["x"]).arrive()
                elif merge:
                    if mistake == "shared exchange":
                        yield lambda: B["wf"][1].passes(w_use[1])
                    else:
                        yield lambda: B["x"].passes(x_use)
                    assert W["pair"] == ("stats", n)
                    W["pair"] = ("weights", n)
                else:
                    W[t] = n
                if merge:
                    x_use += 1
                if not (mistake == "shared exchange" and merge and t == 1):
                    B["wf"][t].arrive()
            B["ie"][n % RING].arrive()
            if nt:
                for c in (0, 1):
                    w_use[c] += both or c == par
                ring_fill += 2 * nt
                par = 0 if two else (par + nt) & 1

    def epilogue():
        use, par = [0, 0], 0
        for n, it in enumerate(seq):
            yield from take(n)
            B["ie"][n % RING].arrive()
            if not it:
                return
            two, nt, n0 = it
            if nt == 0:
                continue
            merge = not two and nt >= 2
            for k in range(2 if two else 1):
                c = k if two else 0 if merge else par
                chains = (0, 1) if merge else (c,)
                for x in chains:
                    yield lambda x=x: B["wf"][x].passes(use[x])
                assert (W["pair"] == ("weights", n)) if merge else W[c] == n
                for x in chains:
                    B["we"][x].arrive()
                for x in chains:
                    yield lambda x=x: B["of"][x].passes(use[x])
                for x in chains:
                    tiles = [(n, j) for j in range(nt) if two and (x == 1 or j < n0) or not two and (par + j) & 1 == x]
                    assert O[x] == tiles, (O[x], tiles)
                    O[x] = []
                done[(n, k)] = True
                yield None
                for x in chains:
                    B["oe"][x].arrive()
            for x in (0, 1):
                use[x] += two or merge or x == par
            par = 0 if two else (par + nt) & 1

    mc.run({"scheduler": scheduler(), "producer": producer(), "loader": loader(), "mma": mma(), "softmax0": softmax(0),
            "softmax1": softmax(1), "epilogue": epilogue()})
    want = {(n, k) for n, it in enumerate(items) if it[1] for k in range(2 if it[0] else 1)}
    assert set(done) == want and not O[0] and not O[1]


def forward_items(rng, n):
    out = []
    for _ in range(n):
        nt = rng.choice([0, 1, 1, 2, 2, 3, 5])
        two = rng.random() < 0.5
        out.append((two, nt, rng.choice([nt, max(1, nt - 1)]) if nt else 0))
    return out


@pytest.mark.parametrize("stages", [5, 8])  # d = 128 and 64
def test_forward_protocol(stages):
    for seed in range(150):
        rng = random.Random(seed)
        forward(rng, forward_items(rng, rng.randrange(1, 24)), stages)


def test_forward_mistake_is_caught():
    """The pair's exchange over the weights' barrier: chain 0 may be items ahead, and an older phase lets it through."""
    caught = 0
    for seed in range(60):
        rng = random.Random(seed)
        try:
            forward(rng, forward_items(rng, 16), 5, "shared exchange")
        except AssertionError:
            caught += 1
    assert caught > 0


# ------------------------------------------------------------------ gradient
def gradient(rng, items, stages, mistake=None):
    """items: (query blocks, the key tile is not full, the last block is not full)."""
    mc = Machine(rng)
    IR = 4
    B = {"kvf": Bar(1), "kvz": Bar(1), "kvd": Bar(1), "kvr": Bar(3)}
    for n in ("qf", "qe", "st"):
        B[n] = [Bar(1) for _ in range(stages)]
    for n, c in (("sp", 1), ("p", 2), ("ds", 2), ("dse", 1), ("dq", 1), ("dqf", 1)):
        B[n] = [Bar(c), Bar(c)]
    B["if"], B["ie"] = [Bar(1) for _ in range(IR)], [Bar(6) for _ in range(IR)]  # producer, MMA, statistics, two P/dS groups, dQ
    ring, kv, zero, qs, st = [None] * IR, [None], [None], [None] * stages, [None] * stages
    sp, p, ds, dq, smem = [None, None], [[None, None], [None, None]], [[None, None], [None, None]], [None, None], [[None, None], [None, None]]
    dv, got = [], []
    seq = list(items) + [None]

    def take(n):
        yield lambda: B["if"][n % IR].passes(n // IR)
        assert ring[n % IR] == n
        B["ie"][n % IR].arrive()

    def scheduler():
        for n in range(len(seq)):
            if n >= IR:
                yield lambda n=n: B["ie"][n % IR].passes(n // IR - 1)
            ring[n % IR] = n
            B["if"][n % IR].arrive()

    def producer():
        c = used = 0
        for n, it in enumerate(seq):
            yield from take(n)
            if not it or it[0] == 0:
                continue
            if used:
                yield lambda: B["kvd"].passes(used - 1)

            def land(n=n):
                kv[0], zero[0] = n, None
                B["kvf"].arrive()

            mc.copies.append(land)
            used += 1
            for i in range(it[0]):
                s = c % stages
                yield lambda s=s, c=c: B["qe"][s].passes(c // stages - 1)

                def land_q(s=s, tag=(n, i)):
                    qs[s] = [tag, False]
                    B["qf"][s].arrive()

                mc.copies.append(land_q)
                c += 1

    def statistics():
        c = used = 0
        for n, it in enumerate(seq):
            yield from take(n)
            if not it or it[0] == 0:
                continue
            if it[1] or mistake != "zero without step":
                yield lambda: B["kvf"].passes(used)
            if it[1]:
                assert kv[0] == n
                zero[0] = n
                B["kvz"].arrive()
            used += 1
            for i in range(it[0]):
                s = c % stages
                yield lambda s=s, c=c: B["qe"][s].passes(c // stages - 1)
                st[s] = (n, i)
                if it[2] and i == it[0] - 1:
                    yield lambda s=s, c=c: B["qf"][s].passes(c // stages)
                    assert qs[s][0] == (n, i)
                    qs[s][1] = True
                B["st"][s].arrive()
                c += 1

    def mma():
        cnt = used = tails = 0

        def issue(n, it, i):
            c = cnt + i
            s, b = c % stages, c & 1
            tail = it[2] and i == it[0] - 1
            yield lambda: B["qf"][s].passes(c // stages)
            if tail:
                yield lambda: B["st"][s].passes(c // stages)

            def scores():
                assert kv[0] == n and (not it[1] or zero[0] == n) and qs[s][0] == (n, i) and qs[s][1] == bool(tail)
                assert p[b] == [None, None], "scores over a P that is still to be read"

            mc.mma.append(scores)
            if c >= 2:
                yield lambda: B["dqf"][b].passes((c - 2) // 2)

            def dp():
                assert dq[b] is None, "dP over a dQ that is still to be read"
                sp[b] = (n, i)
                B["sp"][b].arrive()

            mc.mma.append(dp)

        for n, it in enumerate(seq):
            yield from take(n)
            if not it or it[0] == 0:
                continue
            yield lambda: B["kvf"].passes(used)
            if it[1]:
                yield lambda: B["kvz"].passes(tails)
                tails += 1
            for i in range(min(2, it[0])):
                yield from issue(n, it, i)
            for i in range(it[0]):
                c = cnt + i
                s, b = c % stages, c & 1
                yield lambda: B["p"][b].passes(c // 2)
                if i == 0 and used:
                    yield lambda: B["kvr"].passes(used - 1)

                def add_v(n=n, i=i, b=b, s=s):
                    assert p[b] == [(n, i)] * 2 and qs[s][0] == (n, i)
                    if i == 0:
                        assert not dv, "dV and dK not read yet"
                    dv.append((n, i))
                    p[b] = [None, None]

                mc.mma.append(add_v)
                yield lambda: B["ds"][b].passes(c // 2)

                def add_k(n=n, i=i, b=b, s=s):
                    assert ds[b] == [(n, i)] * 2 and smem[b] == [(n, i)] * 2 and kv[0] == n and qs[s][0] == (n, i)
                    ds[b] = [None, None]
                    dq[b] = (n, i)
                    smem[b] = [None, None]
                    B["dq"][b].arrive()
                    B["dse"][b].arrive()
                    B["qe"][s].arrive()

                mc.mma.append(add_k)
                if i == it[0] - 1:
                    mc.mma.append(B["kvd"].arrive)
                if i + 2 < it[0]:
                    yield from issue(n, it, i + 2)
            cnt += it[0]
            used += 1

    def compute(g):
        c = used = 0
        for n, it in enumerate(seq):
            yield from take(n)
            if not it or it[0] == 0:
                continue
            for i in range(it[0]):
                s, b = c % stages, c & 1
                yield lambda: B["sp"][b].passes(c // 2)
                yield lambda: B["st"][s].passes(c // stages)
                assert sp[b] == (n, i) and st[s] == (n, i)
                p[b][g] = (n, i)
                B["p"][b].arrive()
                yield lambda: B["dse"][b].passes(c // 2 - 1)
                assert sp[b] == (n, i) and st[s] == (n, i) and smem[b][g] is None
                ds[b][g] = smem[b][g] = (n, i)
                B["ds"][b].arrive()
                c += 1
            yield lambda: B["kvd"].passes(used)
            assert dv == [(n, i) for i in range(it[0])]
            yield None
            B["kvr"].arrive()
            used += 1

    def readout():
        c = used = 0
        for n, it in enumerate(seq):
            yield from take(n)
            if not it or it[0] == 0:
                continue
            for i in range(it[0]):
                b = c & 1
                yield lambda: B["dq"][b].passes(c // 2)
                assert dq[b] == (n, i)
                dq[b] = None
                got.append((n, i))
                B["dqf"][b].arrive()
                c += 1
            yield lambda: B["kvd"].passes(used)
            assert dv == [(n, i) for i in range(it[0])]
            yield None
            B["kvr"].arrive()
            used += 1

    # dV and dK are read by three groups: they are gone when the last of them has
    inner = B["kvr"].arrive

    def read():
        inner()
        if B["kvr"].pending == B["kvr"].count:
            dv.clear()

    B["kvr"].arrive = read
    mc.run({"scheduler": scheduler(), "producer": producer(), "statistics": statistics(), "mma": mma(), "compute0": compute(0),
            "compute1": compute(1), "readout": readout()})
    assert got == [(n, i) for n, it in enumerate(items) for i in range(it[0])]


def gradient_items(rng, n):
    return [(rng.choice([0, 1, 1, 2, 3, 4, 7]), rng.random() < 0.4, rng.random() < 0.4) for _ in range(n)]


@pytest.mark.parametrize("stages", [3, 4])  # d = 128 and 64
def test_gradient_protocol(stages):
    for seed in range(150):
        rng = random.Random(seed)
        gradient(rng, gradient_items(rng, rng.randrange(1, 16)), stages)


def test_gradient_mistake_is_caught():
    """Rows zeroed without following every copy of K and V: the copy before lets the wait through."""
    caught = 0
    for seed in range(100):
        rng = random.Random(seed)
        try:
            gradient(rng, gradient_items(rng, 14), 3, "zero without step")
        except AssertionError:
            caught += 1
    assert caught > 0
