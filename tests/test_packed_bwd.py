"""Gradients of attention over packed sequences (attn_bwd_packed) against their formulas in 64 bits, and against
differences of the forward's definition."""
import math

import pytest
import torch

import exact_long_sequence_gb300 as ela
from packed_ref import check_bwd, packed, packed_bwd, starts

pytestmark = pytest.mark.gpu


def rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(ql, kl=None, Hq=4, Hk=2, d=64, causal=True, scale=None, seed=0, tail=3, first=0, token_major=True):
    """As in the forward's tests: tokens of no sequence hold NaN, and their rows of the gradients stay as they were."""
    g = torch.Generator("cuda").manual_seed(seed)
    qs, ks = starts(ql, first), starts(ql if kl is None else kl, first)
    Nq, Nk = qs[-1] + tail, ks[-1] + tail

    def tensor(h, n):
        return rand(g, n, h, d).transpose(0, 1) if token_major else rand(g, h, n, d)

    q, k, v, do = tensor(Hq, Nq), tensor(Hk, Nk), tensor(Hk, Nk), tensor(Hq, Nq)
    for x, end in ((q, qs[-1]), (k, ks[-1]), (v, ks[-1]), (do, qs[-1])):
        x[:, :first], x[:, end:] = math.nan, math.nan
    scale = ela.default_scale(d) if scale is None else scale
    qd, kd = dev(qs), None if kl is None else dev(ks)
    o, lse = ela.attn_fwd_packed(q, k, v, qd, kd, causal=causal, scale=scale)
    out = [torch.full_like(x, 7) for x in (q, k, v)]
    got = ela.attn_bwd_packed(q, k, v, o, lse, do, qd, kd, causal=causal, scale=scale, dq=out[0], dk=out[1], dv=out[2])
    assert ela.last_device_error() == ela.ATTN_OK
    check_bwd(got, *packed_bwd(q, k, v, o, lse, do, qs, ks, causal, scale))
    for x, (a, b) in zip(got, ((qs[0], qs[-1]), (ks[0], ks[-1]), (ks[0], ks[-1]))):
        assert bool((x[:, :a] == 7).all()) and bool((x[:, b:] == 7).all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("ql", [[1], [5], [16, 17], [63, 64, 65], [127, 128, 129], [256, 1, 0, 255], [0, 0, 3, 0], [513, 40], [1000]])
def test_lengths(ql, causal, d):
    run(ql, d=d, causal=causal, seed=sum(ql))


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 3), (3, 1), (5, 1), (6, 2), (7, 1), (16, 2), (24, 2), (32, 1), (64, 1)])
def test_head_groups(Hq, Hk):
    run([70, 1, 300, 33], Hq=Hq, Hk=Hk, d=128, seed=Hq)
    run([70, 1, 300, 33], Hq=Hq, Hk=Hk, d=64, causal=False, seed=Hq)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("ql,kl", [
    ([4, 1, 7], [100, 333, 7]),
    ([300, 2], [20, 0]),
    ([600, 130, 3], [0, 129, 1]),
    ([1, 1, 1, 1], [1, 128, 129, 2000]),
    ([512, 64], [2000, 3001]),
    ([0, 9, 0], [40, 9, 3]),
])
def test_queries_and_keys_apart(ql, kl, causal):
    for d in (64, 128):
        run(ql, kl, Hq=6, Hk=2, d=d, causal=causal, seed=len(ql))


def test_many_sequences():
    g = torch.Generator().manual_seed(3)
    run(torch.randint(0, 40, (400,), generator=g).tolist(), Hq=2, Hk=1, d=64)
    run(torch.randint(0, 300, (70,), generator=g).tolist(), Hq=8, Hk=2, d=128, causal=False)


@pytest.mark.parametrize("scale", [0.0, -0.1, 0.3])
def test_scales(scale):
    run([200, 3, 65], scale=scale, d=64)
    run([200, 3, 65], scale=scale, d=128, causal=False)


def test_contiguous_heads_first_and_offsets():
    run([130, 260, 1], d=128, token_major=False, first=5)
    run([130, 260, 1], d=64, first=1, tail=0)


def test_long():
    run([4000, 100, 2500], Hq=8, Hk=2, d=128, tail=0)
    run([3000, 100, 2500], Hq=3, Hk=3, d=64, causal=False, tail=0)


def test_other_sequences_do_not_reach():
    """NaN and infinities in one sequence leave the gradients of the others within their bounds."""
    d, ql = 64, [37, 130, 65, 1, 128]
    g = torch.Generator("cuda").manual_seed(2)
    qs = starts(ql)
    q, k, v, do = (rand(g, h, qs[-1], d) for h in (4, 2, 2, 4))
    scale = ela.default_scale(d)
    o, lse = ela.attn_fwd_packed(q, k, v, dev(qs), causal=True)
    ref, tol = packed_bwd(q, k, v, o, lse, do, qs, qs, True, scale)
    for s in range(len(ql)):
        own = slice(qs[s], qs[s + 1])
        bad = [x.clone() for x in (q, k, v, do)]
        for x, what in zip(bad, (math.nan, math.inf, math.nan, math.inf)):
            x[:, own] = what
        o2, l2 = ela.attn_fwd_packed(*bad[:3], dev(qs), causal=True)
        got = ela.attn_bwd_packed(*bad[:3], o2, l2, bad[3], dev(qs), causal=True)
        clean = [r.clone() for r in ref]
        for r in clean:
            r[:, own] = math.nan
        check_bwd(got, clean, tol)


def test_against_differences():
    """Along random directions: the gradient's product with a direction is the difference of the loss there, of the
    definition in 64 bits.  The kernel's gradient is off by at most its bound's product with the direction's size."""
    d, ql, kl = 64, [40, 3, 130], [50, 3, 131]
    g = torch.Generator("cuda").manual_seed(8)
    qs, ks = starts(ql), starts(kl)
    q, k, v, do = rand(g, 4, qs[-1], d), rand(g, 2, ks[-1], d), rand(g, 2, ks[-1], d), rand(g, 4, qs[-1], d)
    scale = ela.default_scale(d)
    o, lse = ela.attn_fwd_packed(q, k, v, dev(qs), dev(ks), causal=True)
    got = ela.attn_bwd_packed(q, k, v, o, lse, do, dev(qs), dev(ks), causal=True)
    _, tol = packed_bwd(q, k, v, o, lse, do, qs, ks, True, scale)
    exact_o, _, _ = packed(q, k, v, qs, ks, True, scale)
    loss = lambda a, b, c: (packed(a, b, c, qs, ks, True, scale)[0] * do.double()).sum().item()  # noqa: E731
    base = [q.double(), k.double(), v.double()]
    # D comes from the rounded O: moves dS by P * scale * |dO . (O - exact O)|, and through it dQ and dK
    shift = (do.double() * (o.double() - exact_o)).sum(-1).abs().max().item() * scale
    for which in range(3):
        w = torch.randn(base[which].shape, generator=g, device="cuda", dtype=torch.float64)
        eps = 1e-4
        ends = []
        for sign in (1, -1):
            at = list(base)
            at[which] = base[which] + sign * eps * w
            ends.append(loss(*at))
        slope = (ends[0] - ends[1]) / (2 * eps)
        mine = (got[which].double() * w).sum().item()
        # independent roundings: their products with random directions add up as squares (six sigma)
        room = 6 * (tol[which] ** 2).sum().sqrt().item() + 1e-5 * abs(slope)
        if which < 2:
            other = (k if which == 0 else q).double()
            room += 6 * shift * other.norm(dim=-1).max().item() * math.sqrt(got[which].shape[0] * got[which].shape[1] * (4 if which else 1))
        assert abs(mine - slope) <= room, (which, mine, slope, room)


def test_same_bits_of_dk_and_dv():
    g = torch.Generator("cuda").manual_seed(9)
    qs = starts([700, 33, 401])
    q, k, v, do = (rand(g, h, qs[-1], 128) for h in (6, 2, 2, 6))
    o, lse = ela.attn_fwd_packed(q, k, v, dev(qs), causal=True)
    first = ela.attn_bwd_packed(q, k, v, o, lse, do, dev(qs), causal=True)
    for _ in range(3):
        again = ela.attn_bwd_packed(q, k, v, o, lse, do, dev(qs), causal=True)
        assert torch.equal(first[1], again[1]) and torch.equal(first[2], again[2])


def test_as_attn_bwd_on_equal_lengths():
    B, H, N, d = 3, 4, 257, 128
    g = torch.Generator("cuda").manual_seed(5)
    q, k, v, do = (rand(g, B, H, N, d) for _ in range(4))
    o, lse = ela.attn_fwd(q, k, v, causal=True)
    grads = ela.attn_bwd(q, k, v, o, lse, do, causal=True)
    pack = lambda x: x.transpose(0, 1).reshape(H, B * N, *x.shape[3:])  # noqa: E731
    st = starts([N] * B)
    args = [pack(x).contiguous() for x in (q, k, v, o, lse, do)]
    ref, tol = packed_bwd(*args, st, st, True, ela.default_scale(d))
    check_bwd(ela.attn_bwd_packed(*args, dev(st), causal=True), ref, tol)
    check_bwd([pack(x) for x in grads], ref, tol)


def test_graph_of_both_directions_with_other_lengths():
    d, N = 64, 700
    g = torch.Generator("cuda").manual_seed(6)
    q, k, v, do = (rand(g, h, N, d) for h in (6, 2, 2, 6))
    st = dev([0, 300, 700, 700])
    o, lse = torch.zeros_like(q), torch.zeros((6, N), device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    ws = torch.empty(max(ela.packed_workspace_bytes(3, N, N, 6, 2, d), ela.packed_bwd_workspace_bytes(3, N, N, 6, 2, d)),
                     dtype=torch.uint8, device="cuda")

    def step():
        ela.attn_fwd_packed(q, k, v, st, causal=True, out=o, lse=lse, workspace=ws)
        ela.attn_bwd_packed(q, k, v, o, lse, do, st, causal=True, dq=dq, dk=dk, dv=dv, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for ql in ([300, 400, 0], [1, 1, 1], [0, 0, 700], [450, 249, 1]):
        qs = starts(ql)
        st.copy_(dev(qs))
        for x in (dq, dk, dv):
            x.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        check_bwd((dq, dk, dv), *packed_bwd(q, k, v, o, lse, do, qs, qs, True, ela.default_scale(d)))
        for x in (dq, dk, dv):
            assert bool((x[:, qs[-1]:] == 7).all())
