"""Attention of new tokens over a paged cache (attn_fwd_tree) against its definition in 64 bits."""
import math

import pytest
import torch

import exact_long_sequence_gb300 as ela
from packed_ref import bits, check, tree

pytestmark = pytest.mark.gpu


def rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cache(g, lens, page, Hk, d, token_major, spare=2):
    """Pages in a random order; what is no request's key holds NaN.  Returns K, V, the table (its unused entries bad)."""
    need = [max(0, (n + page - 1) // page) for n in lens]
    total = sum(need) + spare
    if token_major:
        k, v = (rand(g, total, page, Hk, d).transpose(1, 2) for _ in range(2))
    else:
        k, v = (rand(g, total, Hk, page, d) for _ in range(2))
    ids = torch.randperm(total, generator=g, device="cuda").tolist()
    table = torch.full((len(lens), max(1, max(need))), 1 << 30, dtype=torch.int32)
    used = torch.zeros((total, page), dtype=torch.bool)
    for r, n in enumerate(lens):
        for i in range(need[r]):
            pg = ids.pop()
            table[r, i] = pg
            used[pg, : min(page, n - i * page)] = True
    hole = ~used.cuda()[:, None, :, None].expand_as(k)
    for x in (k, v):
        x.masked_fill_(hole, math.nan)
    return k, v, table.cuda()


def random_tree(g, R, T):
    """Every token follows one of those before it, or the last cached token."""
    seen = torch.zeros((R, T, T), dtype=torch.bool)
    for r in range(R):
        for t in range(T):
            parent = int(torch.randint(-1, t, (1,), generator=g)) if t else -1
            if parent >= 0:
                seen[r, t] = seen[r, parent]
            seen[r, t, t] = True
    return seen.cuda()


def run(lens, T=1, Hq=4, Hk=2, d=64, page=16, token_major=True, mask="tree", scale=None, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    R = len(lens)
    kc, vc, table = cache(g, lens, page, Hk, d, token_major)
    q = rand(g, R, T, Hq, d).transpose(1, 2)
    scale = ela.default_scale(d) if scale is None else scale
    if mask == "tree":
        seen = random_tree(torch.Generator().manual_seed(seed), R, T)
    elif mask == "random":
        seen = torch.rand((R, T, T), generator=g, device="cuda") < 0.3
    elif mask == "nothing":
        seen = torch.zeros((R, T, T), dtype=torch.bool, device="cuda")
    else:
        seen = torch.ones((T, T), dtype=torch.bool, device="cuda").tril().expand(R, T, T)
    out, lse = torch.full((R, T, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2), torch.full((R, Hq, T), 7.0, device="cuda")
    words = None if mask is None else bits(seen).cuda()
    if words is not None and T % 32:
        words[..., -1] |= -1 << (T % 32)  # bits past T do not count
    ela.attn_fwd_tree(q, kc, vc, table, dev(lens), words, scale=scale, out=out, lse=lse)
    assert ela.last_device_error() == ela.ATTN_OK
    check(out, lse, tree(q, kc, vc, table, lens, seen, scale))
    pad = torch.tensor([n < 0 for n in lens], device="cuda")
    assert bool((out[pad] == 7).all()) and bool((lse[pad] == 7).all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
def test_single_tokens(page, d):
    run([1, 2, 15, 16, 17, 127, 128, 129, 500, 1025], page=page, d=d, mask=None, seed=page)
    run([1, 2, 15, 16, 17, 127, 128, 129, 500, 1025], page=page, d=d, token_major=False, seed=page)


@pytest.mark.parametrize("mask", ["tree", "random", "nothing", None])
@pytest.mark.parametrize("T", [2, 5, 16, 31, 32, 33, 64, 70, 129])
def test_drafts(T, mask):
    run([T, T + 1, T + 100, 300 + T, 128, 640], T=T, mask=mask, d=128 if T % 2 else 64, seed=T)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 1), (5, 1), (7, 1), (8, 8), (16, 2), (48, 2), (64, 1)])
def test_head_groups(Hq, Hk):
    for T in (1, 9, 24):
        run([T, 200, 77], T=T, Hq=Hq, Hk=Hk, d=128, page=32, seed=T)


@pytest.mark.parametrize("T", [1, 6])
def test_empty_and_padded_requests(T):
    run([0, -1, 40, -5, 0, 1, T], T=T, mask="tree")
    run([-1, -1], T=T, mask="tree")
    run([0], T=T, mask=None)
    run([1, 2, 3], T=6, mask=None)       # fewer keys than new tokens: the first new ones are missing
    run([1, 2, 3], T=6, mask="random")
    run([0, 0, 0], T=6, mask="nothing")


def test_many_requests():
    g = torch.Generator().manual_seed(0)
    run(torch.randint(-1, 300, (700,), generator=g).tolist(), Hq=4, Hk=2, d=64, mask=None)
    run(torch.randint(8, 900, (60,), generator=g).tolist(), T=8, Hq=8, Hk=4, d=128, page=64)


def test_long():
    run([40000, 9, 20011], T=8, Hq=8, Hk=2, d=128, page=128)
    run([70001], T=1, Hq=8, Hk=1, d=64, page=16, mask=None)


@pytest.mark.parametrize("scale", [0.0, -0.1, 0.4])
def test_scales(scale):
    run([5, 200, 131], T=5, scale=scale)


def test_table_longer_than_needed_and_lens_past_it():
    g = torch.Generator("cuda").manual_seed(1)
    kc, vc, table = cache(g, [64, 48], 16, 2, 64, True)
    wide = torch.full((2, 9), -3, dtype=torch.int32, device="cuda")
    wide[:, :4] = table
    q = rand(g, 2, 4, 1, 64)
    seen = torch.ones((2, 1, 1), dtype=torch.bool, device="cuda")
    out, lse = ela.attn_fwd_tree(q, kc, vc, wide[:, :4], dev([64, 48]))  # rows 9 apart
    check(out, lse, tree(q, kc, vc, table, [64, 48], seen, ela.default_scale(64)))
    out, lse = ela.attn_fwd_tree(q, kc, vc, table[:, :2].contiguous(), dev([1 << 30, 30]))
    check(out, lse, tree(q, kc, vc, table[:, :2], [32, 30], seen, ela.default_scale(64)))


def test_pages_outside_the_cache_read_as_zeros():
    g = torch.Generator("cuda").manual_seed(2)
    kc, vc = rand(g, 3, 1, 16, 64), rand(g, 3, 1, 16, 64)
    q = rand(g, 1, 1, 1, 64)
    zero = torch.zeros_like(kc[:1])
    for bad in (-1, 3, 1 << 30, -(1 << 31)):
        out, lse = ela.attn_fwd_tree(q, kc, vc, dev([[1, bad, 2]]), dev([41]))
        assert ela.last_device_error() == ela.ATTN_OK
        ref = tree(q, torch.cat([kc, zero]), torch.cat([vc, zero]), dev([[1, 3, 2]]), [41],
                   torch.ones((1, 1, 1), dtype=torch.bool, device="cuda"), ela.default_scale(64))
        check(out, lse, ref)


def test_a_hidden_draft_does_not_reach():
    """NaN in the K of a drafted token reaches only the tokens that see it."""
    g = torch.Generator("cuda").manual_seed(3)
    T, n = 6, 150
    kc, vc, table = cache(g, [n], 16, 1, 64, False)
    q = rand(g, 1, 2, T, 64)
    seen = random_tree(torch.Generator().manual_seed(9), 1, T)
    clean, lse0 = ela.attn_fwd_tree(q, kc, vc, table, dev([n]), bits(seen).cuda())
    for j in range(T):
        key = n - T + j
        k2 = kc.clone()
        k2[table[0, key // 16], :, key % 16] = math.nan
        out, lse = ela.attn_fwd_tree(q, k2, vc, table, dev([n]), bits(seen).cuda())
        hit = seen[0, :, j]
        assert torch.equal(out[0, :, ~hit], clean[0, :, ~hit]) and torch.equal(lse[0, :, ~hit], lse0[0, :, ~hit])
        assert bool(torch.isnan(out[0, :, hit].float()).all())


def test_graph_with_other_lengths_and_trees():
    g = torch.Generator("cuda").manual_seed(4)
    R, T = 3, 7
    most = [200, 333, 90]
    kc, vc, table = cache(g, most, 32, 2, 128, True)
    kc.nan_to_num_(0.0)
    vc.nan_to_num_(0.0)
    q = rand(g, R, 8, T, 128)
    lens, words = dev(most), bits(random_tree(torch.Generator().manual_seed(0), R, T)).cuda()
    out, lse = torch.zeros_like(q), torch.zeros((R, 8, T), device="cuda")
    ws = torch.empty(ela.tree_workspace_bytes(R, 8, 2, T, 128), dtype=torch.uint8, device="cuda")
    ela.attn_fwd_tree(q, kc, vc, table, lens, words, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ela.attn_fwd_tree(q, kc, vc, table, lens, words, out=out, lse=lse, workspace=ws)
    for i, new in enumerate(([200, 333, 90], [7, 64, 33], [-1, 300, 8])):
        seen = random_tree(torch.Generator().manual_seed(i), R, T)
        lens.copy_(dev(new))
        words.copy_(bits(seen))
        graph.replay()
        torch.cuda.synchronize()
        check(out, lse, tree(q, kc, vc, table, new, seen, ela.default_scale(128)))
