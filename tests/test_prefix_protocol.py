"""Models of the shared-prefix attention's host-free parts, on the CPU.

1. The cut of the work (csrc/attn_prefix_kernel.cuh: the scheduler warp, OwnCut; csrc/attn_prefix_api.cu:
   lay_out, the workspace): every tile of every row block is taken exactly once, every piece
   has partial rows of its own inside the workspace, and the combine kernel reads exactly the pieces
   that were written.
2. The barrier protocol of the roles of one CTA, replayed under many random interleavings with the
   kernel's arrival counts and issue order, as the forward kernel's model does: no deadlock, no barrier
   two phases ahead of a waiter, and every buffer (K/V stages, query slots, score and output
   accumulators, the exchanged statistics) holds what its reader expects when it is read.
   An asynchronous operation completes at once here, the most permissive timing for run-ahead.
Like the kernel's own documentation, the models state it; when the kernel changes, they change with it.
"""
import random

import pytest

TILE, ITEM, BC, BR = 4, 2, 128, 128
STAGES, RING = 5, 8


# ------------------------------------------------------------------ 1. the cut
def cdiv(a, b):
    return -(-a // b)


class PrefixCut:
    """The cut of the prefix's tiles into stretches, the first `early` of a run longer."""

    def __init__(self, Hk, ptiles, psegs, early, lead, own_total):
        self.Hk, self.ptiles, self.psegs, self.early = Hk, ptiles, psegs, early
        self.by_head = psegs % Hk == 0
        self.len = ptiles if self.by_head else ptiles * Hk
        self.per = psegs // Hk if self.by_head else psegs
        assert 0 <= early < self.per <= self.len
        self.etiles = self.ebase = self.erem = 0
        self.lbase, self.lrem = divmod(self.len, self.per)
        if early:
            ahead = min(self.len, early * (own_total * lead >> 20))
            late = (self.len - ahead) // self.per
            self.etiles = self.len - late * (self.per - early)
            self.ebase, self.erem = divmod(self.etiles, early)
            self.lbase, self.lrem = late, 0

    def run_begin(self, i):
        if i < self.early:
            return i * self.ebase + min(i, self.erem)
        return self.etiles + (i - self.early) * self.lbase + min(i - self.early, self.lrem)

    def place(self, k):
        if not self.by_head:
            return 0, k
        first = self.early * self.Hk
        n, y = (self.early, k) if k < first else (self.per - self.early, k - first)
        return y // n, y % n + (0 if k < first else self.early)

    def begin(self, k, past):
        run, i = self.place(k)
        return run * self.len + self.run_begin(i + past)

    def run_of(self, y):
        if y < self.etiles:
            longer = self.erem * (self.ebase + 1)
            return y // (self.ebase + 1) if y < longer else self.erem + (y - longer) // self.ebase
        y -= self.etiles
        longer = self.lrem * (self.lbase + 1)
        return self.early + (y // (self.lbase + 1) if y < longer else self.lrem + (y - longer) // self.lbase)

    def slot(self, k, head):
        return head * self.per + self.place(k)[1] if self.by_head else k + head

    def head_slots(self, h):
        """Where the combine kernel looks for a head's pieces."""
        base = 0 if self.by_head else h * self.ptiles
        i0 = self.run_of(base)
        n = self.run_of(base + self.ptiles - 1) - i0 + 1
        return [(h * self.per if self.by_head else h) + i0 + i for i in range(n)]


@pytest.mark.parametrize("seed", range(12))
def test_the_cut_of_the_prefix(seed):
    """Every tile once, every piece in a slot of its own, and the slots that are read are those written."""
    rng = random.Random(seed)
    for _ in range(60):
        Hk, ptiles = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 7, 19, 64, 200])
        psegs = rng.choice([n for n in (1, 2, 3, 5, 8, 16, 19, 24, 38, 64, 152) if n <= Hk * ptiles])
        per = psegs // Hk if psegs % Hk == 0 else psegs
        early = rng.randrange(per)
        c = PrefixCut(Hk, ptiles, psegs, early, rng.choice([0, 891, 1 << 20]), rng.choice([0, 1, 500, 20000, 1 << 29]))
        seen, slots = set(), {}
        for k in range(psegs):
            x, end = c.begin(k, 0), c.begin(k, 1)
            assert x <= end
            while x < end:
                head = x // ptiles
                n = min(end - x, (head + 1) * ptiles - x)
                tiles = set(range(x, x + n))
                assert not tiles & seen and c.slot(k, head) not in slots
                assert 0 <= c.slot(k, head) < psegs + (0 if c.by_head else Hk - 1)
                seen |= tiles
                slots[c.slot(k, head)] = head
                x += n
        assert seen == set(range(Hk * ptiles))
        for h in range(Hk):
            read = c.head_slots(h)
            assert len(set(read)) == len(read) and set(read) == {s for s, head in slots.items() if head == h}


class Layout:
    def __init__(self, R, Hk, G, T, P, C, grid):
        self.R, self.Hk, self.GT, self.T, self.P, self.C, self.grid = R, Hk, G * T, T, P, C, grid
        self.ptiles = cdiv(P, BC)
        self.two = 2 * (128 // self.GT * self.GT if self.GT <= 128 else 128)  # rows of two query tiles
        self.pblocks, self.oblocks = cdiv(R * self.GT, self.two), cdiv(self.GT, self.two)
        self.orows = min(self.GT, self.two)
        self.psegs, self.pitems = 0, 0
        self.line = Hk * self.ptiles
        if self.ptiles:
            most = min(max(2 * grid // self.pblocks, 8), self.line)
            best = None
            for n in range(1, most + 1):
                pieces = 1 if n % Hk == 0 else cdiv(Hk, n) + 1
                cost = (cdiv(self.pblocks * n, grid) * (cdiv(self.line, n) * TILE + pieces * 8.0) +
                        4.2e-4 * R * self.GT * (n + Hk))
                if best is None or cost < best:
                    best, self.psegs = cost, n
            self.pitems = self.pblocks * self.psegs
            self.cut = PrefixCut(Hk, self.ptiles, self.psegs, 0, 0, 0)
        by_head = self.psegs % Hk == 0
        self.own_first = (self.psegs + (0 if by_head else Hk - 1)) * R * self.GT if self.psegs else 0
        self.rows = self.own_first + ((R * Hk * self.oblocks + grid) * self.orows if C else 0)

    def seq_cost(self, n):
        return ITEM + cdiv(n, 32) if n > 0 else 0


class Cut:
    def __init__(self, L, total):
        g = L.grid
        self.rem = L.pitems % g
        item = ITEM + cdiv(L.line, L.psegs) * TILE if L.psegs else 0
        level = item * (g - self.rem)
        if self.rem == 0 or total > level:
            e = cdiv(total - (0 if self.rem == 0 else level), g)
            self.cap1, self.cap0 = e, e if self.rem == 0 else item + e
        else:
            self.cap1, self.cap0 = 0, cdiv(total, g - self.rem)
        if 0 < self.cap1 < TILE:
            self.cap1 = TILE
        self.cap0 = max(self.cap0, TILE)

    def begin(self, b):
        return b * self.cap1 if b < self.rem else self.rem * self.cap1 + (b - self.rem) * self.cap0

    def cta_of(self, x):
        return x // self.cap1 if x < self.rem * self.cap1 else self.rem + (x - self.rem * self.cap1) // self.cap0


def schedule(L, lens, cta):
    """The items of one CTA: (req, head, row0, nrows, tile0, ntiles, first partial row)."""
    out = []
    for i in range(cta, L.pitems, L.grid):
        blk, k = i % L.pblocks, i // L.pblocks
        row0 = blk * L.two
        x, end = L.cut.begin(k, 0), L.cut.begin(k, 1)
        assert x < end
        while x < end:
            head = x // L.ptiles
            t0 = x - head * L.ptiles
            n = min(end - x, L.ptiles - t0)
            out.append((-1, head, row0, min(L.two, L.R * L.GT - row0), t0, n,
                        L.cut.slot(k, head) * L.R * L.GT + row0))
            x += n
    if not L.C:
        return out
    lens = [min(max(n, 0), L.C) for n in lens]
    seqs = L.Hk * L.oblocks
    run = cdiv(L.R, 32)
    mine = [sum(L.seq_cost(n) * seqs for n in lens[k * run:(k + 1) * run]) for k in range(32)]
    upto = [sum(mine[:k + 1]) for k in range(32)]
    cut = Cut(L, upto[31])
    x0, x1 = cut.begin(cta), min(cut.begin(cta + 1), upto[31])
    if x0 >= x1:
        return out
    at = next(k for k in range(32) if upto[k] > x0)
    start = upto[at] - mine[at]
    for r in range(at * run, L.R):
        if start >= x1:
            break
        cost = L.seq_cost(lens[r])
        if lens[r] > 0 and start + cost * seqs > x0:
            nt = cdiv(lens[r], BC)
            for q in range((x0 - start) // cost if x0 > start else 0, seqs):
                if start + q * cost >= x1:
                    break
                first = start + q * cost + ITEM
                t0 = min(cdiv(x0 - first, TILE) if x0 > first else 0, nt)
                t1 = min(cdiv(x1 - first, TILE) if x1 > first else 0, nt)
                if t0 >= t1:
                    continue
                blk = q % L.oblocks
                out.append((r, q // L.oblocks, r * L.GT + blk * L.two, min(L.two, L.GT - blk * L.two), t0, t1 - t0,
                            L.own_first + (r * seqs + q + cta) * L.orows))
        start += cost * seqs
    return out


def combine_rows(L, lens, r, h, x):
    """The partial rows the combine kernel merges for row x of request r at key head h."""
    rows = []
    if L.ptiles:
        rows = [slot * L.R * L.GT + r * L.GT + x for slot in L.cut.head_slots(h)]
    n = min(lens[r], L.C) if L.C else 0
    if n > 0:
        seqs = L.Hk * L.oblocks
        starts = [0]
        for v in lens:
            starts.append(starts[-1] + L.seq_cost(min(max(v, 0), L.C)) * seqs)
        cut = Cut(L, starts[-1])
        q = h * L.oblocks + x // L.two
        first = starts[r] + q * L.seq_cost(n) + ITEM
        a, b = cut.cta_of(first), cut.cta_of(first + (n - 1) // BC * TILE)
        rows += [L.own_first + (r * seqs + q + c) * L.orows + x % L.two for c in range(a, b + 1)]
    return rows


def own_lengths(kind, R, C, rng):
    return {"zero": lambda: 0, "full": lambda: C, "one": lambda: 1, "padding": lambda: rng.choice([-1, 0, 1, C]),
            "any": lambda: rng.randint(-1, C + 5), "few": lambda: rng.choice([0] * 9 + [C])}[kind]()


@pytest.mark.parametrize("kind", ["zero", "full", "one", "padding", "any", "few"])
@pytest.mark.parametrize("R,Hk,G,T,P,C,grid", [
    (1, 1, 1, 1, 1, 0, 152), (1, 1, 1, 1, 0, 5, 152), (3, 2, 4, 1, 1000, 700, 152), (5, 1, 3, 100, 300, 900, 8),
    (70, 2, 2, 1, 0, 4000, 152), (33, 8, 4, 2, 5000, 257, 152), (2, 4, 1, 300, 129, 400, 11), (100, 3, 1, 1, 128, 31, 13),
    (1, 1, 64, 1, 70000, 50000, 152), (40, 1, 16, 1, 2048, 129, 7),
])
def test_every_tile_once_and_every_piece_found(R, Hk, G, T, P, C, grid, kind):
    rng = random.Random(R * 31 + P)
    L = Layout(R, Hk, G, T, P, C, grid)
    lens = [own_lengths(kind, R, C, rng) for _ in range(R)]
    tiles, written = {}, set()
    for cta in range(grid):
        for req, head, row0, nrows, t0, nt, part in schedule(L, lens, cta):
            assert nt >= 1 and 1 <= nrows <= 256
            for j in range(t0, t0 + nt):
                key = (req, head, row0, j)
                assert key not in tiles
                tiles[key] = cta
            span = set(range(part, part + nrows))
            assert not span & written and 0 <= part and part + nrows <= L.rows
            written |= span
    want = {(-1, h, b * L.two, j) for h in range(Hk) for b in range(L.pblocks) for j in range(L.ptiles)}
    for r in range(R):
        for h in range(Hk):
            for b in range(L.oblocks):
                want |= {(r, h, r * L.GT + b * L.two, j) for j in range(cdiv(min(max(lens[r], 0), C), BC))}
    assert set(tiles) == want
    read = set()
    for r in range(R):
        for h in range(Hk):
            for x in range(L.GT):
                rows = combine_rows(L, lens, r, h, x)
                assert len(set(rows)) == len(rows) and not read & set(rows) and set(rows) <= written
                read |= set(rows)
    assert read == written  # nothing computed for nothing, padding's prefix rows included


# The own-keys kernel's cut (requests with few rows a key head): steps of 16 keys, one stretch a warp.
# Hk stands for a request's sequences: key heads times row blocks.
def warp_seq_cost(n):
    return 1 + cdiv(n, 16) if n > 0 else 0


def warp_walk(R, Hk, lens, total, upto, mine, run, worker, workers):
    """(request, key head, first step, end) of every piece of a warp, by the kernel's walk."""
    cap = max(1, cdiv(total, workers))
    x0, x1 = worker * cap, min(worker * cap + cap, total)
    out = []
    if x0 >= x1:
        return out
    at = next(k for k in range(32) if upto[k] > x0)
    r, start, h = at * run, upto[at] - mine[at], 0
    while r < R and start + warp_seq_cost(lens[r]) * Hk <= x0:
        start += warp_seq_cost(lens[r]) * Hk
        r += 1
    cost = warp_seq_cost(lens[r]) if r < R else 0
    if cost:
        h = (x0 - start) // cost
        start += h * cost
    while start < x1 and r < R:
        cost = warp_seq_cost(lens[r])
        if lens[r] > 0 and start + cost > x0:
            s, s1 = max(0, x0 - start - 1), min(x1 - start - 1, cost - 1)
            if s < s1:
                out.append((r, h, s, s1))
        start += cost
        h += 1
        if lens[r] == 0 or h == Hk:
            r, h = r + 1, 0
    return out


@pytest.mark.parametrize("kind", ["zero", "full", "one", "padding", "any", "few"])
@pytest.mark.parametrize("R,Hk,C,workers", [(1, 1, 1, 6), (1, 8, 5000, 912), (3, 2, 700, 912), (70, 2, 400, 60), (33, 8, 33, 912),
                                            (200, 1, 17, 912), (100, 3, 31, 18), (40, 4, 129, 912)])
def test_every_own_step_once_and_every_piece_found(R, Hk, C, workers, kind):
    rng = random.Random(R * 31 + C)
    lens = [min(max(own_lengths(kind, R, C, rng), 0), C) for _ in range(R)]
    run = cdiv(R, 32)
    mine = [Hk * sum(warp_seq_cost(n) for n in lens[k * run:(k + 1) * run]) for k in range(32)]
    upto = [sum(mine[:k + 1]) for k in range(32)]
    total = upto[31]
    steps, slots = set(), set()
    for w in range(workers):
        for r, h, s, s1 in warp_walk(R, Hk, lens, total, upto, mine, run, w, workers):
            assert s < s1
            for j in range(s, s1):
                assert (r, h, j) not in steps
                steps.add((r, h, j))
            slot = r * Hk + h + w
            assert slot not in slots and slot < R * Hk + workers
            slots.add(slot)
    assert steps == {(r, h, j) for r in range(R) for h in range(Hk) for j in range(cdiv(lens[r], 16))}
    cap, at, read = max(1, cdiv(total, workers)), 0, set()
    for r in range(R):
        for h in range(Hk):
            if lens[r] > 0:
                first = at + h * warp_seq_cost(lens[r]) + 1
                read |= {r * Hk + h + w for w in range(first // cap, (first + (lens[r] - 1) // 16) // cap + 1)}
        at += warp_seq_cost(lens[r]) * Hk
    assert read == slots


# ------------------------------------------------------------------ 2. the barriers
class Barrier:
    def __init__(self, name, count):
        self.name, self.count, self.pending, self.done = name, count, count, 0

    def arrive(self, n=1):
        self.pending -= n
        assert self.pending >= 0, f"{self.name}: more arrivals than the count"
        if self.pending == 0:
            self.done += 1
            self.pending = self.count


def run(items, seed, stages=STAGES, o_empty_twice=True):
    """One CTA over items (two query tiles?, K/V tiles, zeroed tail?).  None, or what went wrong."""
    rng = random.Random(seed)
    B = {}

    def mk(name, count=1):
        B[name] = Barrier(name, count)

    for s in range(stages):
        mk(("KvFull", s)), mk(("KvEmpty", s))
    for t in (0, 1):
        for n in ("QFull", "QEmpty", "SFull", "OFull"):
            mk((n, t))
        mk(("PHalf", t), 128), mk(("PFull", t), 128), mk(("OEmpty", t), 256), mk(("X", t), 128)
    for s in range(RING):
        mk(("ItemFull", s)), mk(("ItemEmpty", s), 11)
    stage, qslot, S, O = [None] * stages, [None] * 2, [None] * 2, [None] * 2
    xchg = [None]
    entries = items + [None]
    slot_item = [None] * RING

    def need(got, want, what):
        if got != want:
            raise AssertionError(f"{what}: {got}, wanted {want}")

    def take(n):
        yield ("ItemFull", n % RING), n // RING
        need(slot_item[n % RING], n, "item")

    def scheduler():
        for n in range(len(entries)):
            if n >= RING:
                yield ("ItemEmpty", n % RING), n // RING - 1
            slot_item[n % RING] = n
            B[("ItemFull", n % RING)].arrive()

    def producer():
        pos = 0
        for n, it in enumerate(entries):
            yield from take(n)
            B[("ItemEmpty", n % RING)].arrive()
            if it is None:
                return
            for j in range(it[1]):
                for kv in "KV":
                    st, use = pos % stages, pos // stages
                    if use:
                        yield ("KvEmpty", st), use - 1
                    stage[st] = (n, kv, j)
                    B[("KvFull", st)].arrive()
                    pos += 1

    def qloader():
        qpos = 0
        for n, it in enumerate(entries):
            yield from take(n)
            B[("ItemEmpty", n % RING)].arrive()
            if it is None:
                return
            for k in range(2 if it[0] else 1):
                if qpos >= 2:
                    yield ("QEmpty", qpos & 1), (qpos >> 1) - 1
                qslot[qpos & 1] = (n, k)
                B[("QFull", qpos & 1)].arrive()
                qpos += 1

    def mma():
        kpos = qpos = par = 0
        pph, oph = [0, 0], [0, 0]
        due = []

        def run_pv():
            if not due:
                return
            n, j, c, k, v, first, last, first_v, last_v = due.pop()
            if first_v:
                yield ("KvFull", v % stages), v // stages
            yield ("PHalf", c), pph[c]
            if first:
                if oph[c]:
                    yield ("OEmpty", c), oph[c] - 1
                oph[c] += 1
                O[c] = [n, k, []]
            need(S[c], ("P", n, j, k), "P half")
            yield ("PFull", c), pph[c]
            pph[c] += 1
            need(S[c], ("P", n, j, k), "P")
            need(stage[v % stages], (n, "V", j), "V")
            need(O[c][:2], [n, k], "O")
            O[c][2].append(j)
            if last_v:
                B[("KvEmpty", v % stages)].arrive()
            if last:
                B[("OFull", c)].arrive()

        def free(c):  # the score buffer of the product that ran (unless the next scores already went into it)
            if S[c][0] == "P":
                S[c] = ("free",)

        def pv_now():
            if due:
                c = due[0][2]
                yield from run_pv()
                free(c)

        for n, it in enumerate(entries):
            if rng.random() < 0.3:  # the next item is not known yet: the due product goes first
                yield from pv_now()
            yield from take(n)
            B[("ItemEmpty", n % RING)].arrive()
            if it is None:
                break
            two, nt, _ = it
            steps = 2 * nt if two else nt
            par = 0 if two else par
            for s in range(steps):
                j, k = (s >> 1, s & 1) if two else (s, 0)
                c = (par + s) & 1
                if due and (due[0][2] == c or ((s == 0 or not two) and rng.random() < 0.3)):
                    assert due[0][2] != c or (two and s == 0)  # the same chain again: only at a two-tile item's start
                    yield from pv_now()  # or its operands are not there yet
                if k == 0:
                    yield ("KvFull", kpos % stages), kpos // stages
                if j == 0:
                    yield ("QFull", (qpos + k) & 1), (qpos + k) >> 1
                need(stage[kpos % stages], (n, "K", j), "K")
                need(qslot[(qpos + k) & 1], (n, k), "Q")
                last_k = not two or k == 1
                if S[c] is not None:
                    need(S[c][0], "free", "score buffer still in use")
                S[c] = ("S", n, j, k)
                B[("SFull", c)].arrive()
                if last_k:
                    B[("KvEmpty", kpos % stages)].arrive()
                if j == nt - 1:
                    B[("QEmpty", (qpos + k) & 1)].arrive()
                yield from pv_now()
                due.append((n, j, c, k, kpos + 1, j == 0 if two else s < 2, j == nt - 1 if two else s + 2 >= steps,
                            k == 0, last_k))
                if last_k:
                    kpos += 2
            qpos += 2 if two else 1
            par = 0 if two else (par + steps) & 1
        yield from run_pv()

    def softmax(t):
        s_cnt = x_cnt = ring = par = 0
        o_cnt = [0, 0]
        for n, it in enumerate(entries):
            yield from take(n)
            if it is None:
                return
            two, nt, tail = it
            steps = 2 * nt if two else nt
            mine = t if two else t ^ par
            k = mine if two else 0
            both = two or nt >= 2
            if both or mine == 0:
                js = range(nt) if two else range(mine, nt, 2)
                for j in js:
                    yield ("SFull", t), s_cnt
                    s_cnt += 1
                    need(S[t], ("S", n, j, k), "S")
                    if tail and k == 0 and j == nt - 1:
                        at = ring + 2 * j + 1
                        yield ("KvFull", at % stages), at // stages
                        need(stage[at % stages], (n, "V", j), "V to be zeroed")
                    S[t] = ("P", n, j, k)
                    B[("PHalf", t)].arrive(128)
                    yield None
                    B[("PFull", t)].arrive(128)
                yield ("OFull", t), o_cnt[t]
                need(O[t], [n, k, list(js)], "finished O")
                if both and not two:
                    if t == 1:
                        xchg[0] = (n, 1)
                        B[("X", 1)].arrive(128)
                    yield ("X", t ^ 1), x_cnt
                    yield ("OFull", t ^ 1), o_cnt[t ^ 1]
                    need(xchg[0], (n, t ^ 1), "other chain's statistics")
                    if t == 0:
                        xchg[0] = (n, 0)
                        B[("X", 0)].arrive(128)
                    x_cnt += 1
                    need(O[t ^ 1], [n, 0, list(range(1 - mine, nt, 2))], "other chain's O")
                    yield None
                    need(O[t ^ 1], [n, 0, list(range(1 - mine, nt, 2))], "other chain's O after the readout")
                    B[("OEmpty", 0)].arrive(128)
                    B[("OEmpty", 1)].arrive(128)
                else:
                    B[("OEmpty", t)].arrive(256 if o_empty_twice else 128)
            for c in (0, 1):
                if both or par == c:
                    o_cnt[c] += 1
            ring += 2 * nt
            par = 0 if two else (par + steps) & 1
            need(slot_item[n % RING], n, "the item at its end")
            B[("ItemEmpty", n % RING)].arrive(4)

    roles = {"scheduler": scheduler(), "producer": producer(), "qloader": qloader(), "mma": mma(), "softmax0": softmax(0),
             "softmax1": softmax(1)}
    waiting = {k: None for k in roles}
    alive = set(roles)
    while alive:
        runnable = []
        for k in sorted(alive):
            w = waiting[k]
            if w is None:
                runnable.append(k)
                continue
            done = B[w[0]].done
            if done >= w[1] + 2:
                return f"phase overrun: {k} waits {w[0]} phase {w[1]}, barrier already completed {done}"
            if done >= w[1] + 1:
                runnable.append(k)
        if not runnable:
            return f"deadlock: { {k: waiting[k] for k in sorted(alive)} }"
        k = rng.choice(runnable)
        waiting[k] = None
        try:
            waiting[k] = next(roles[k])
        except StopIteration:
            alive.discard(k)
        except AssertionError as e:
            return f"{k}: {e}"
    return None


ITEMS = [
    [(False, 1, False)], [(True, 1, True)], [],
    [(False, 1, True)] * 9,
    [(False, 7, False), (False, 2, True), (False, 1, True), (False, 1, False), (False, 3, True)],
    [(True, 5, False), (False, 4, False), (True, 1, False), (False, 1, True), (True, 2, True)],
    [(False, 2, True)] * 7, [(True, 3, False)] * 4 + [(False, 1, True)] * 6,
]


@pytest.mark.parametrize("items", ITEMS + [[(random.Random(k).random() < 0.3, random.Random(k + i).randint(1, 4),
                                             random.Random(k * i).random() < 0.5) for i in range(12)] for k in range(8)])
def test_protocol(items):
    for seed in range(25):
        assert run(items, seed) is None
        assert run(items, seed, stages=8) is None


def test_checker_finds_an_accumulator_that_is_never_released():
    found = [run([(False, 1, False)] * 6, seed, o_empty_twice=False) for seed in range(5)]
    assert all(f and f.startswith("deadlock") for f in found)
