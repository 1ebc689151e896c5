"""Attention over packed sequences (attn_fwd_packed) against its definition in 64 bits."""
import math

import pytest
import torch

import exact_long_sequence_gb300 as ela
from packed_ref import check, packed, starts

pytestmark = pytest.mark.gpu


def rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(ql, kl=None, Hq=4, Hk=2, d=64, causal=True, scale=None, seed=0, tail=3, first=0, token_major=True):
    """Sequences of these lengths, with `first` tokens before and `tail` behind them that belong to none; what is not a
    sequence's holds NaN, and rows of no sequence must stay as they were."""
    g = torch.Generator("cuda").manual_seed(seed)
    kl_ = ql if kl is None else kl
    qs, ks = starts(ql, first), starts(kl_, first)
    Nq, Nk = qs[-1] + tail, ks[-1] + tail
    if token_major:
        q, k, v = (rand(g, n, h, d).transpose(0, 1) for n, h in ((Nq, Hq), (Nk, Hk), (Nk, Hk)))
    else:
        q, k, v = rand(g, Hq, Nq, d), rand(g, Hk, Nk, d), rand(g, Hk, Nk, d)
    for x in (k, v):
        x[:, :first], x[:, ks[-1]:] = math.nan, math.nan
    out, lse = torch.full((Nq, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1), torch.full((Hq, Nq), 7.0, device="cuda")
    scale = ela.default_scale(d) if scale is None else scale
    ela.attn_fwd_packed(q, k, v, dev(qs), None if kl is None else dev(ks), causal=causal, scale=scale, out=out, lse=lse)
    assert ela.last_device_error() == ela.ATTN_OK
    check(out, lse, packed(q, k, v, qs, ks, causal, scale))
    outside = torch.ones(Nq, dtype=torch.bool, device="cuda")
    outside[qs[0]:qs[-1]] = False
    assert bool((out[:, outside] == 7).all()) and bool((lse[:, outside] == 7).all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("ql", [[1], [5], [16, 17], [127, 128, 129], [256, 1, 0, 255], [0, 0, 3, 0], [513, 40], [1000]])
def test_lengths(ql, causal, d):
    run(ql, d=d, causal=causal, seed=sum(ql))


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 3), (3, 1), (5, 1), (6, 2), (7, 1), (16, 2), (24, 2), (32, 1), (64, 1)])
def test_head_groups(Hq, Hk):
    run([70, 1, 300, 33], Hq=Hq, Hk=Hk, d=128, seed=Hq)
    run([70, 1, 300, 33], Hq=Hq, Hk=Hk, d=64, causal=False, seed=Hq)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("ql,kl", [
    ([4, 1, 7], [100, 333, 7]),            # new tokens behind others' keys
    ([300, 2], [20, 0]),                   # more queries than keys, and none: causal rows that see nothing
    ([600, 130, 3], [0, 129, 1]),
    ([1, 1, 1, 1], [1, 128, 129, 5000]),   # single tokens
    ([512, 64], [5000, 9001]),
    ([0, 9, 0], [40, 9, 3]),
])
def test_queries_and_keys_apart(ql, kl, causal):
    for d in (64, 128):
        run(ql, kl, Hq=6, Hk=2, d=d, causal=causal, seed=len(ql))


def test_many_sequences():
    g = torch.Generator().manual_seed(3)
    run(torch.randint(0, 40, (1000,), generator=g).tolist(), Hq=2, Hk=1, d=64)
    run(torch.randint(0, 300, (70,), generator=g).tolist(), Hq=8, Hk=2, d=128, causal=False)


@pytest.mark.parametrize("scale", [0.0, -0.1, 0.5, 1e-30])
def test_scales(scale):
    run([200, 3, 65], scale=scale, d=64)
    run([200, 3, 65], scale=scale, d=128, causal=False)


def test_contiguous_heads_first_and_offsets():
    run([130, 260, 1], d=128, token_major=False, first=5)
    run([130, 260, 1], d=64, token_major=True, first=1, tail=0)


def test_long():
    run([6000, 100, 2500], Hq=8, Hk=2, d=128, tail=0)
    run([3000, 100, 2500], Hq=3, Hk=3, d=64, causal=False, tail=0)


def test_one_key_decides():
    """A key whose score is far above the others', wherever it lies, takes the row; late ones move the reference."""
    d, n = 128, 700
    g = torch.Generator("cuda").manual_seed(1)
    q, k, v = rand(g, 2, 2 * n, d), rand(g, 1, 2 * n, d), rand(g, 1, 2 * n, d)
    qs = [0, n, 2 * n]
    for at in (0, 15, 16, 127, 128, 255, 300, 511, 699):
        kk = k.clone()
        q2 = q.clone()
        q2[:, :, 0] = 8
        kk[:, [at, n + at], :] = 0
        kk[:, [at, n + at], 0] = 256  # score 2048 / sqrt(128) = 181 for the rows that see it
        out, lse = ela.attn_fwd_packed(q2, kk, v, dev(qs), causal=True)
        check(out, lse, packed(q2, kk, v, qs, qs, True, ela.default_scale(d)))


def test_other_sequences_do_not_reach():
    """NaN and infinities in one sequence's K and V leave the others as they are, bit for bit."""
    d, ql = 64, [37, 130, 65, 1, 128]
    g = torch.Generator("cuda").manual_seed(2)
    qs = starts(ql)
    q, k, v = rand(g, 4, qs[-1], d), rand(g, 2, qs[-1], d), rand(g, 2, qs[-1], d)
    clean, clean_lse = ela.attn_fwd_packed(q, k, v, dev(qs), causal=True)
    for s in range(len(ql)):
        k2, v2, q2 = k.clone(), v.clone(), q.clone()
        own = slice(qs[s], qs[s + 1])
        k2[:, own], v2[:, own], q2[:, own] = math.nan, math.inf, math.nan
        out, lse = ela.attn_fwd_packed(q2, k2, v2, dev(qs), causal=True)
        rest = torch.ones(qs[-1], dtype=torch.bool, device="cuda")
        rest[own] = False
        assert torch.equal(out[:, rest], clean[:, rest]) and torch.equal(lse[:, rest], clean_lse[:, rest])
        assert bool(torch.isnan(out[:, own].float()).all())


def test_bad_offsets_are_clipped():
    d = 64
    g = torch.Generator("cuda").manual_seed(4)
    q, k, v = rand(g, 2, 100, d), rand(g, 2, 90, d), rand(g, 2, 90, d)
    qs, ks = [-5, 40, 30, 60, 2000], [0, 1 << 30, -7, 90, 95]
    clip = lambda x, n: min(max(x, 0), n)  # noqa: E731
    out, lse = torch.full_like(q, 7), torch.full((2, 100), 7.0, device="cuda")
    ela.attn_fwd_packed(q, k, v, dev(qs), dev(ks), out=out, lse=lse)
    assert ela.last_device_error() == ela.ATTN_OK
    check(out, lse, packed(q, k, v, [clip(x, 100) for x in qs], [clip(x, 90) for x in ks], False, ela.default_scale(d)))


def test_as_attn_fwd_on_equal_lengths():
    """The same sequences through attn_fwd: both within their bounds of the same definition."""
    B, H, N, d = 3, 4, 257, 128
    g = torch.Generator("cuda").manual_seed(5)
    q, k, v = (rand(g, B, H, N, d) for _ in range(3))
    o, lse = ela.attn_fwd(q, k, v, causal=True)
    pack = lambda x: x.transpose(0, 1).reshape(H, B * N, d)  # noqa: E731
    out, l2 = ela.attn_fwd_packed(pack(q), pack(k), pack(v), dev(starts([N] * B)), causal=True)
    ref = packed(pack(q), pack(k), pack(v), starts([N] * B), starts([N] * B), True, ela.default_scale(d))
    check(out, l2, ref)
    check(pack(o), lse.transpose(0, 1).reshape(H, B * N), ref)


def test_graph_with_other_lengths():
    d, Nq = 128, 900
    g = torch.Generator("cuda").manual_seed(6)
    q, k, v = rand(g, 8, Nq, d), rand(g, 2, Nq, d), rand(g, 2, Nq, d)
    st = dev([0, 300, 900, 900])
    out, lse = torch.zeros_like(q), torch.zeros((8, Nq), device="cuda")
    ws = torch.empty(ela.packed_workspace_bytes(3, Nq, Nq, 8, 2, d), dtype=torch.uint8, device="cuda")
    ela.attn_fwd_packed(q, k, v, st, causal=True, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ela.attn_fwd_packed(q, k, v, st, causal=True, out=out, lse=lse, workspace=ws)
    for ql in ([300, 600, 0], [1, 1, 1], [0, 0, 900], [450, 449, 1]):
        qs = starts(ql)
        st.copy_(dev(qs))
        out.fill_(7)
        lse.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        check(out, lse, packed(q, k, v, qs, qs, True, ela.default_scale(d)))
        assert bool((out[:, qs[-1]:] == 7).all())
        first = out.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, out)


def test_another_stream():
    d = 64
    g = torch.Generator("cuda").manual_seed(7)
    q, k, v = rand(g, 4, 500, d), rand(g, 2, 500, d), rand(g, 2, 500, d)
    qs = [0, 123, 500]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = ela.attn_fwd_packed(q, k, v, dev(qs), causal=True, stream=s)
    s.synchronize()
    check(out, lse, packed(q, k, v, qs, qs, True, ela.default_scale(d)))
