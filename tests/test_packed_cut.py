"""Packed and paged calls whose units are cut for certain: masks of several words, head groups of any size, scales, and
values that must not reach other rows, in pieces and in their merge (GPU).

Up to 640 keys in all, or with few keys to a row, units are left whole; so that a case here does not become such a
call unnoticed, each asserts that the call left cuts at the head of its workspace ([stretches] records of eight words, the first
the number of pieces).
"""
import math

import pytest
import torch

import exact_long_sequence_gb300 as ela
from packed_ref import bits, check, packed, starts, tree
from test_tree import cache, dev, rand, random_tree

pytestmark = pytest.mark.gpu


def assert_cut(ws):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert int(ws[:32 * sms].view(torch.int32).view(-1, 8)[:, 0].max()) > 1


def packed_call(q, k, v, qs, ks, causal=True, scale=None):
    ws = torch.zeros(ela.packed_workspace_bytes(len(qs) - 1, q.shape[1], k.shape[1], q.shape[0], k.shape[0], q.shape[2]),
                     dtype=torch.uint8, device="cuda")
    got = ela.attn_fwd_packed(q, k, v, dev(qs), dev(ks), causal=causal, scale=scale, workspace=ws)
    assert ela.last_device_error() == ela.ATTN_OK
    assert_cut(ws)
    return got


def tree_call(q, kc, vc, table, lens, words, scale=None):
    R, Hq, T, d = q.shape
    ws = torch.zeros(ela.tree_workspace_bytes(R, Hq, kc.shape[1], T, d), dtype=torch.uint8, device="cuda")
    got = ela.attn_fwd_tree(q, kc, vc, table, dev(lens), words, scale=scale, workspace=ws)
    assert ela.last_device_error() == ela.ATTN_OK
    assert_cut(ws)
    return got


def run_tree(lens, T, Hq, Hk, d, page, mask, scale=None, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    R = len(lens)
    kc, vc, table = cache(g, lens, page, Hk, d, seed % 2 == 0)
    q = rand(g, R, T, Hq, d).transpose(1, 2)
    if mask == "tree":
        seen = random_tree(torch.Generator().manual_seed(seed), R, T)
    elif mask == "random":
        seen = torch.rand((R, T, T), generator=g, device="cuda") < 0.3
    elif mask == "nothing":
        seen = torch.zeros((R, T, T), dtype=torch.bool, device="cuda")
    else:
        seen = torch.ones((T, T), dtype=torch.bool, device="cuda").tril().expand(R, T, T)
    words = None if mask is None else bits(seen).cuda()
    if words is not None and T % 32:
        words[..., -1] |= -1 << (T % 32)  # bits past T do not count
    scale = ela.default_scale(d) if scale is None else scale
    out, lse = tree_call(q, kc, vc, table, lens, words, scale)
    check(out, lse, tree(q, kc, vc, table, lens, seen, scale))


@pytest.mark.parametrize("mask", ["tree", "random", "nothing", None])
@pytest.mark.parametrize("T", [31, 32, 33, 64, 70, 129])
def test_drafts(T, mask):
    run_tree([3000 + T, 20000, 9011], T, 4, 2, 128 if T % 2 else 64, 64, mask, seed=T)


@pytest.mark.parametrize("shift", [1, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128])
def test_new_tokens_across_a_tile(shift):
    """The new tokens begin `shift` keys before a tile's end, so that a mask's words straddle tiles and chunks."""
    run_tree([128 * 40 - shift + 70, 128 * 30 - shift + 70], 70, 6, 2, 64, 16, "random", seed=shift)


@pytest.mark.parametrize("G", [1, 3, 5, 7, 48, 64])
@pytest.mark.parametrize("T", [1, 9, 40])
def test_head_groups_of_drafts(T, G):
    run_tree([20011, T, 200, 77], T, 2 * G, 2, 128 if G % 2 else 64, 32, "tree", seed=G)
    run_tree([9000, 40 + T], T, G, 1, 64 if G % 2 else 128, 128, None, seed=G + 1)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("G", [1, 3, 5, 7, 48, 64])
def test_head_groups_of_packed_sequences(G, causal):
    ql, kl = [70, 1, 300, 33, 0, 5], [9001, 1, 300, 700, 20, 2]
    for d in (64, 128):
        g = torch.Generator("cuda").manual_seed(G)
        qs, ks = starts(ql), starts(kl)
        q, k, v = rand(g, qs[-1], 2 * G, d).transpose(0, 1), rand(g, 2, ks[-1], d), rand(g, ks[-1], 2, d).transpose(0, 1)
        out, lse = packed_call(q, k, v, qs, ks, causal)
        check(out, lse, packed(q, k, v, qs, ks, causal, ela.default_scale(d)))


@pytest.mark.parametrize("scale", [0.0, -0.1, 0.4, 1e-30])
def test_scales(scale):
    run_tree([20000, 5000, 131], 33, 4, 2, 64, 16, "random", scale=scale)
    qs, ks = starts([200, 3, 65]), starts([7000, 3, 4001])
    g = torch.Generator("cuda").manual_seed(1)
    q, k, v = rand(g, 6, qs[-1], 128), rand(g, 2, ks[-1], 128), rand(g, 2, ks[-1], 128)
    for causal in (False, True):
        out, lse = packed_call(q, k, v, qs, ks, causal, scale)
        check(out, lse, packed(q, k, v, qs, ks, causal, scale))


def test_other_sequences_do_not_reach():
    d, qs, ks = 64, starts([37, 130, 65, 1, 128]), starts([3000, 2007, 900, 4001, 2600])
    g = torch.Generator("cuda").manual_seed(2)
    q, k, v = rand(g, 4, qs[-1], d), rand(g, 2, ks[-1], d), rand(g, 2, ks[-1], d)
    clean, clean_lse = packed_call(q, k, v, qs, ks)
    for s in range(len(qs) - 1):
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        own, keys = slice(qs[s], qs[s + 1]), slice(ks[s], ks[s + 1])
        k2[:, keys], v2[:, keys], q2[:, own] = math.nan, math.inf, math.nan
        out, lse = packed_call(q2, k2, v2, qs, ks)
        rest = torch.ones(qs[-1], dtype=torch.bool, device="cuda")
        rest[own] = False
        assert torch.equal(out[:, rest], clean[:, rest]) and torch.equal(lse[:, rest], clean_lse[:, rest])
        assert bool(torch.isnan(out[:, own].float()).all()) and bool(torch.isnan(lse[:, own]).all())


def test_a_hidden_draft_does_not_reach():
    """NaN in the K of a drafted token reaches only the tokens that see it, over two words of a mask."""
    g = torch.Generator("cuda").manual_seed(3)
    T, n = 40, 5003
    kc, vc, table = cache(g, [n], 16, 1, 64, False)
    q = rand(g, 1, 2, T, 64)
    seen = random_tree(torch.Generator().manual_seed(9), 1, T)
    words = bits(seen).cuda()
    clean, lse0 = tree_call(q, kc, vc, table, [n], words)
    for j in (0, 1, 12, 31, 32, 39):
        key = n - T + j
        k2 = kc.clone()
        k2[table[0, key // 16], :, key % 16] = math.nan
        out, lse = tree_call(q, k2, vc, table, [n], words)
        hit = seen[0, :, j]
        assert torch.equal(out[0, :, ~hit], clean[0, :, ~hit]) and torch.equal(lse[0, :, ~hit], lse0[0, :, ~hit])
        assert bool(torch.isnan(out[0, :, hit].float()).all())


def test_one_key_decides():
    """A key whose score is far above the others', in any of the pieces, takes the rows that see it."""
    d, n, m = 128, 40, 9000
    g = torch.Generator("cuda").manual_seed(1)
    q, k, v = rand(g, 2, n, d), rand(g, 1, m, d), rand(g, 1, m, d)
    q[:, :, 0] = 8
    for at in (0, 127, 128, 1000, 4500, 8831, 8832, 8959, 8960, 8970, 8999):
        k2 = k.clone()
        k2[:, at] = 0
        k2[:, at, 0] = 256  # score 2048 / sqrt(128) = 181
        out, lse = packed_call(q, k2, v, [0, n], [0, m])
        check(out, lse, packed(q, k2, v, [0, n], [0, m], True, ela.default_scale(d)))
