"""Query / key preparation (head norm and rotary positions) and its gradient: refusals and the
reference's own gradient on the CPU, parity with the 64-bit formulas on the GPU (bounds: see
qk_norm_rope_ref)."""
import ctypes

import numpy as np
import pytest
import torch

import exact_long_sequence_gb300 as ela
from exact_long_sequence_gb300 import _build

import qk_norm_rope_ref as ref

gpu = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ela.load_library()


def cdll_call(lib, fn="fwd", **over):
    """The C entry with plausible addresses, `over` replacing arguments by name."""
    s3 = ctypes.c_int64 * 3
    a = dict(Q=0x1000, qs=None, K=0x2000, ks=None, wq=0x3000, wk=0x4000, pos=0x5000, pa=0, pb=0, inv=0x6000,
             sec=(16, 16), Qo=0x7000, qos=None, Ko=0x8000, kos=None, B=2, Hq=4, Hk=2, N=8, d=64, eps=EPS, inter=0,
             g=0x9000, gs=None, gk=0xA000, gks=None, dwq=0xB000, dwk=0xC000, ws=0xD000, wsb=1 << 24)
    a.update(over)
    for k in ("qs", "ks", "qos", "kos", "gs", "gks"):
        a[k] = s3(*a[k]) if a[k] is not None else None
    n = len(a["sec"]) if a["sec"] is not None else 1
    sec = (ctypes.c_int * max(n, 1))(*a["sec"]) if a["sec"] is not None else None
    shape = (a["B"], a["Hq"], a["Hk"], a["N"], a["d"], a["eps"], a["inter"])
    if fn == "fwd":
        return lib.attn_qk_norm_rope(a["Q"], a["qs"], a["K"], a["ks"], a["wq"], a["wk"], a["pos"], a["pa"], a["pb"],
                                     a["inv"], sec, n, a["Qo"], a["qos"], a["Ko"], a["kos"], *shape, None)
    return lib.attn_qk_norm_rope_bwd(a["g"], a["gs"], a["gk"], a["gks"], a["Q"], a["qs"], a["K"], a["ks"], a["wq"],
                                     a["wk"], a["pos"], a["pa"], a["pb"], a["inv"], sec, n, a["Qo"], a["qos"], a["Ko"],
                                     a["kos"], a["dwq"], a["dwk"], *shape, a["ws"], a["wsb"], None)


BAD = [
    (dict(pos=None), ela.ATTN_ERR_INVALID_ARG), (dict(inv=None), ela.ATTN_ERR_INVALID_ARG),
    (dict(sec=None), ela.ATTN_ERR_INVALID_ARG), (dict(Qo=None), ela.ATTN_ERR_INVALID_ARG),
    (dict(N=0), ela.ATTN_ERR_INVALID_ARG), (dict(B=0), ela.ATTN_ERR_INVALID_ARG), (dict(Hk=0), ela.ATTN_ERR_INVALID_ARG),
    (dict(B=1 << 16, N=1 << 16), ela.ATTN_ERR_INVALID_ARG), (dict(eps=float("nan")), ela.ATTN_ERR_INVALID_ARG),
    (dict(eps=-1e-6), ela.ATTN_ERR_INVALID_ARG), (dict(d=96), ela.ATTN_ERR_UNSUPPORTED),
    (dict(sec=(16, 17)), ela.ATTN_ERR_INVALID_ARG),      # more pairs than d / 2
    (dict(sec=(16, 0, 16)), ela.ATTN_ERR_INVALID_ARG),   # an axis without pairs
    (dict(sec=(8, 8, 8, 4, 4)), ela.ATTN_ERR_INVALID_ARG),  # five axes
    (dict(sec=(12,)), ela.ATTN_ERR_UNSUPPORTED),         # not a multiple of 8 pairs
    (dict(Q=0x1008), ela.ATTN_ERR_MISALIGNED), (dict(wk=0x4008), ela.ATTN_ERR_MISALIGNED),
    (dict(Ko=0x8002), ela.ATTN_ERR_MISALIGNED), (dict(pos=0x5002), ela.ATTN_ERR_MISALIGNED),
    (dict(inv=0x6004), ela.ATTN_ERR_MISALIGNED),
    (dict(qs=(4096, 512, 68)), ela.ATTN_ERR_MISALIGNED),  # a token stride that is not a multiple of 8
    (dict(kos=(1024, 512, 0)), ela.ATTN_ERR_INVALID_ARG),  # written rows on top of one another
]


@pytest.mark.parametrize("fn", ["fwd", "bwd"])
@pytest.mark.parametrize("over,status", BAD)
def test_refusals(lib, fn, over, status):
    assert cdll_call(lib, fn, **over) == status


def test_backward_refusals(lib):
    assert cdll_call(lib, "bwd", g=None) == ela.ATTN_ERR_INVALID_ARG
    assert cdll_call(lib, "bwd", dwq=None) == ela.ATTN_ERR_INVALID_ARG            # a weight without its gradient
    assert cdll_call(lib, "bwd", wk=None) == ela.ATTN_ERR_INVALID_ARG             # and the other way round
    assert cdll_call(lib, "bwd", K=None) == ela.ATTN_ERR_INVALID_ARG              # a norm needs its input
    assert cdll_call(lib, "bwd", ws=None) == ela.ATTN_ERR_INVALID_ARG
    assert cdll_call(lib, "bwd", ws=0xD008) == ela.ATTN_ERR_MISALIGNED
    assert cdll_call(lib, "bwd", dwk=0xC002) == ela.ATTN_ERR_MISALIGNED
    assert lib.attn_qk_norm_rope_bwd_workspace_bytes(96) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_valid_calls_without_gpu_report_no_device(lib):
    none = (ela.ATTN_ERR_NO_DEVICE, ela.ATTN_ERR_CUDA)
    assert cdll_call(lib) in none and cdll_call(lib, wq=None, qs=(0, 512, 64)) in none
    assert cdll_call(lib, B=1, kos=(0, 512, 64)) in none  # the stride of an axis of one is not looked at
    assert cdll_call(lib, "bwd") in none
    assert cdll_call(lib, "bwd", wq=None, wk=None, dwq=None, dwk=None, Q=None, K=None, ws=None, wsb=0) in none


def test_binding_refuses_on_the_host():
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ela.qk_norm_rope(q, q, torch.zeros(4, dtype=torch.int32), torch.ones(32, dtype=torch.float64))


def test_quotients_by_multiplication():
    """The rule the kernels divide token numbers by (struct Quotient), over its whole range of numbers."""
    rng = np.random.default_rng(3)
    divisors = [*range(1, 400), *(2 ** k + e for k in range(9, 31) for e in (-1, 0, 1)), 2 ** 31 - 1]
    for d in divisors + rng.integers(1, 2 ** 31, 300).tolist():
        s = (d - 1).bit_length()
        m = -(-(1 << (31 + s)) // d) if d > 1 else 0
        assert m < 2 ** 32
        ns = np.concatenate([rng.integers(0, 2 ** 31, 50), rng.integers(0, 2 ** 31, 50) // d * d, [0, 2 ** 31 - 1]])
        for n in {int(n) + e for n in ns for e in (-1, 0) if 0 <= n + e < 2 ** 31}:
            assert (n if d == 1 else n * m >> 32 >> (s - 1)) == n // d


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_gradient_against_differences(interleaved):
    rng = np.random.default_rng(5)
    x, dy = rng.standard_normal((2, 2, 3, 3, 64))
    w = 1 + 0.2 * rng.standard_normal(64)
    t = ref.angles(rng.integers(0, 50, (2, 2, 3)), 0.5 ** np.arange(24), (10, 14))
    loss = lambda x, w: (ref.forward(x, w, t, EPS, interleaved)[0] * dy).sum()  # noqa: E731
    dx, _, dw, _ = ref.backward(dy, x, w, t, EPS, interleaved)
    h = 1e-5
    for at in [(0, 0, 0, 0), (1, 2, 2, 63), (1, 0, 1, 30), (0, 1, 2, 50)]:
        e = np.zeros_like(x)
        e[at] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[at]) < 1e-7
    for j in (0, 31, 63):
        e = np.zeros(64)
        e[j] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[j]) < 1e-7


# ------------------------------------------------------------------ GPU
def inputs(B, Hq, Hk, N, d, rot, sections, far, seed, fused=False, spiky=False):
    g = torch.Generator().manual_seed(seed)

    def draw(*shape):
        x = torch.randn(*shape, generator=g)
        if spiky:  # rows of very different size, some all zero
            x = x * 10.0 ** torch.randint(-12, 13, shape[:-1] + (1,), generator=g)
            x = x * (torch.rand(shape[:-1] + (1,), generator=g) > 0.1)
        return x.to(torch.bfloat16).cuda()

    if fused:
        p = draw(B, N, Hq + 2 * Hk, d)
        q, k = p[:, :, :Hq].transpose(1, 2), p[:, :, Hq:Hq + Hk].transpose(1, 2)
    else:
        q, k = draw(B, Hq, N, d), draw(B, Hk, N, d)
    pos = torch.randint(-far if far > 1000 else 0, far + 1, (len(sections), B, N), generator=g, dtype=torch.int64)
    pos = pos.to(torch.int32).cuda()
    inv = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda() for _ in range(2))
    dq, dk = draw(B, Hq, N, d), draw(B, Hk, N, d)
    return q, k, pos, inv.cuda(), wq, wk, dq, dk


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def check_forward(x, w, pos, inv, sections, eps, inter, y):
    t = ref.angles(pos.cpu().numpy(), inv.cpu().numpy(), sections)
    want, S = ref.forward(f64(x), f64(w), t, eps, inter)
    assert np.isfinite(f64(y)).all()
    assert ref.excess(f64(y), want, S) <= 0


def check_backward(dy, x, w, pos, inv, sections, eps, inter, dx, dw):
    t = ref.angles(pos.cpu().numpy(), inv.cpu().numpy(), sections)
    want, S, want_w, Sw = ref.backward(f64(dy), f64(x), f64(w), t, eps, inter)
    assert ref.excess(f64(dx), want, S) <= 0
    if w is None:
        assert dw is None
        return
    rows = x.shape[0] * x.shape[1] * x.shape[2]
    assert dw.dtype == torch.float32
    assert (np.abs(f64(dw) - want_w) <= (2.0 ** -18 + rows * 2.0 ** -24) * Sw + 1e-38).all()


# d, Hq, Hk, B, N, rotated, sections, interleaved, farthest position, fused projection
SHAPES = [
    (64, 1, 1, 1, 1, 64, (32,), False, 0, False),
    (64, 8, 8, 2, 37, 64, (32,), True, 5000, False),
    (64, 9, 3, 3, 5, 32, (3, 13), False, 1000, True),
    (64, 17, 1, 1, 7, 16, (1, 2, 5), True, 1000, True),
    (128, 1, 1, 1, 3, 128, (64,), False, 1 << 20, False),
    (128, 32, 8, 2, 65, 128, (16, 24, 24), False, 300, True),
    (128, 32, 8, 1, 1, 128, (64,), True, (1 << 20), True),
    (128, 5, 5, 2, 33, 96, (7, 40, 1), False, 1000, False),
    (128, 6, 2, 2, 9, 80, (10, 10, 10, 10), True, 1000, True),
    (128, 16, 4, 1, 2500, 128, (64,), False, 2500, True),  # whole tokens per warp
    (128, 2, 1, 3, 333, 128, (20, 20, 24), True, 500, True),  # several tokens per warp step, the last step short
    (64, 3, 2, 5, 501, 48, (24,), False, 500, False),
    (64, 1, 4, 2, 4099, 64, (32,), False, 5000, True),
    (128, 40, 8, 64, 1, 64, (32,), False, 100000, True),
]


@gpu
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_parity(lib, shape, norm):
    d, Hq, Hk, B, N, rot, sections, inter, far, fused = shape
    q, k, pos, inv, wq, wk, dqo, dko = inputs(B, Hq, Hk, N, d, rot, sections, far, seed=N + Hq, fused=fused)
    if not norm:
        wq = wk = None
    kw = dict(q_weight=wq, k_weight=wk, sections=sections, eps=EPS, interleaved=inter)
    qo, ko = ela.qk_norm_rope(q, k, pos, inv, **kw)
    assert qo.shape == q.shape and qo.is_contiguous() and ko.shape == k.shape and ko.is_contiguous()
    check_forward(q, wq, pos, inv, sections, EPS, inter, qo)
    check_forward(k, wk, pos, inv, sections, EPS, inter, ko)
    dq, dk, dwq, dwk = ela.qk_norm_rope_bwd(dqo, dko, q, k, pos, inv, **kw)
    check_backward(dqo, q, wq, pos, inv, sections, EPS, inter, dq, dwq)
    check_backward(dko, k, wk, pos, inv, sections, EPS, inter, dk, dwk)


@gpu
def test_only_one_tensor_has_a_norm_and_one_position_row_serves_every_batch(lib):
    q, k, pos, inv, wq, wk, dqo, dko = inputs(3, 4, 2, 11, 128, 128, (64,), 2000, seed=2)
    row = pos[0, 0].contiguous()
    all_b = row.expand(1, 3, 11)
    kw = dict(k_weight=wk, eps=EPS)
    qo, ko = ela.qk_norm_rope(q, k, row, inv, **kw)
    check_forward(q, None, all_b, inv, (64,), EPS, False, qo)
    check_forward(k, wk, all_b, inv, (64,), EPS, False, ko)
    dq, dk, dwq, dwk = ela.qk_norm_rope_bwd(dqo, dko, q, k, row, inv, **kw)
    check_backward(dqo, q, None, all_b, inv, (64,), EPS, False, dq, dwq)
    check_backward(dko, k, wk, all_b, inv, (64,), EPS, False, dk, dwk)


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_very_different_size_and_zero_rows(lib, d):
    """eps decides for tiny rows; a zero row gives zeros, and its gradient is u w / sqrt(eps)."""
    q, k, pos, inv, wq, wk, dqo, dko = inputs(2, 6, 3, 29, d, d, (d // 2,), 1000, seed=3, spiky=True)
    kw = dict(q_weight=wq, k_weight=wk, eps=EPS)
    qo, ko = ela.qk_norm_rope(q, k, pos, inv, **kw)
    check_forward(q, wq, pos, inv, (d // 2,), EPS, False, qo)
    check_forward(k, wk, pos, inv, (d // 2,), EPS, False, ko)
    dq, dk, dwq, dwk = ela.qk_norm_rope_bwd(dqo, dko, q, k, pos, inv, **kw)
    check_backward(dqo, q, wq, pos, inv, (d // 2,), EPS, False, dq, dwq)
    check_backward(dko, k, wk, pos, inv, (d // 2,), EPS, False, dk, dwk)


@gpu
def test_zero_eps_with_an_odd_number_of_heads(lib):
    """Lanes without a head add nothing to the weights' gradient where eps is 0."""
    q, k, pos, inv, wq, wk, dqo, dko = inputs(1, 3, 1, 5, 128, 128, (64,), 100, seed=4)
    dq, dk, dwq, dwk = ela.qk_norm_rope_bwd(dqo, dko, q, k, pos, inv, q_weight=wq, k_weight=wk, eps=0.0)
    check_backward(dqo, q, wq, pos, inv, (64,), 0.0, False, dq, dwq)
    check_backward(dko, k, wk, pos, inv, (64,), 0.0, False, dk, dwk)


@gpu
def test_nonfinite_rows_stay_in_their_rows(lib):
    q, k, pos, inv, wq, wk, _, _ = inputs(1, 4, 4, 16, 64, 64, (32,), 100, seed=6)
    q[0, 1, 3, 7] = float("nan")
    k[0, 2, 5, 0] = float("inf")
    qo, ko = ela.qk_norm_rope(q, k, pos, inv, q_weight=wq, k_weight=wk)
    bad_q, bad_k = ~torch.isfinite(qo).all(-1), ~torch.isfinite(ko).all(-1)
    assert bad_q.nonzero().tolist() == [[0, 1, 3]] and bad_k.nonzero().tolist() == [[0, 2, 5]]


@gpu
@pytest.mark.parametrize("p", [2 ** 31 - 1, -2 ** 31, 123456789])
def test_the_farthest_positions(lib, p):
    """The reference angle in integers: position * freq for freq = 2 pi k / 2^40 turns is exact modulo a turn."""
    pairs = 32
    k64 = [(987654321987 * (i + 1)) % 2 ** 40 for i in range(pairs)]  # turns per position, times 2^40
    inv = torch.tensor([2 * np.pi * v / 2 ** 40 for v in k64], dtype=torch.float64).cuda()
    x = torch.randn(1, 1, 1, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    pos = torch.tensor([p], dtype=torch.int32).cuda()
    y, _ = ela.qk_norm_rope(x, x, pos, inv)
    t = np.array([2 * np.pi * (((p * v) % 2 ** 40) / 2 ** 40) for v in k64])[None, None, None]
    want, S = ref.forward(f64(x), None, t, EPS, False)
    # the frequency itself is rounded to float64, and its turns to 2^-53: the angle may be off by 2 pi |p| 2^-52
    off = 2 * np.pi * abs(p) * 2.0 ** -52 * S
    assert (np.abs(f64(y) - want) <= off + 2.0 ** -18 * S + 2.0 ** -8 * (np.abs(want) + off + 2.0 ** -18 * S)).all()


@gpu
def test_views_in_place_and_the_rows_of_a_cache(lib):
    q, k, pos, inv, wq, wk, dqo, dko = inputs(2, 4, 2, 6, 128, 128, (64,), 100, seed=7, fused=True)
    kw = dict(q_weight=wq, k_weight=wk, sections=(64,))
    qo, ko = ela.qk_norm_rope(q, k, pos, inv, **kw)
    # rows 3..8 of a cache of 11, the others left as they were; token-major storage
    cache = torch.full((2, 11, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    view = cache.transpose(1, 2)[:, :, 3:9]
    q2 = q.clone(memory_format=torch.contiguous_format)
    ela.qk_norm_rope(q2, k, pos, inv, q_out=q2, k_out=view, **kw)
    assert torch.equal(q2, qo) and torch.equal(view, ko)
    assert (cache[:, :3] == 7.0).all() and (cache[:, 9:] == 7.0).all()
    # gradients into the slices of a fused gradient, in place over the upstream one
    want = ela.qk_norm_rope_bwd(dqo, dko, q, k, pos, inv, **kw)
    grad = torch.full((2, 6, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    got = ela.qk_norm_rope_bwd(dqo, dko, q, k, pos, inv, dq=grad[:, :, :4].transpose(1, 2),
                               dk=grad[:, :, 4:6].transpose(1, 2), **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and (grad[:, :, 6:] == 5.0).all()
    got = ela.qk_norm_rope_bwd(dqo, dko, q, k, pos, inv, dq=dqo, dk=dko, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # one row for every head (a broadcast input)
    one = torch.randn(2, 1, 6, 128, device="cuda").to(torch.bfloat16)
    a, b = ela.qk_norm_rope(one.expand(2, 4, 6, 128), one, pos, inv, **kw)
    a2, _ = ela.qk_norm_rope(one.expand(2, 4, 6, 128).contiguous(), one, pos, inv, **kw)
    assert torch.equal(a, a2)


@gpu
def test_streams_graphs_and_repeated_calls_give_the_same_bits(lib):
    q, k, pos, inv, wq, wk, dqo, dko = inputs(2, 8, 2, 200, 128, 128, (16, 24, 24), 300, seed=8)
    kw = dict(q_weight=wq, k_weight=wk, sections=(16, 24, 24))
    fwd = ela.qk_norm_rope(q, k, pos, inv, **kw)
    bwd = ela.qk_norm_rope_bwd(dqo, dko, q, k, pos, inv, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    f2 = ela.qk_norm_rope(q, k, pos, inv, stream=side, **kw)
    b2 = ela.qk_norm_rope_bwd(dqo, dko, q, k, pos, inv, stream=side, **kw)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(fwd + bwd, f2 + b2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f3 = ela.qk_norm_rope(q, k, pos, inv, **kw)
        b3 = ela.qk_norm_rope_bwd(*f3, q, k, pos, inv, **kw)
    q.copy_(q.roll(1, 2))
    graph.replay()
    f4 = ela.qk_norm_rope(q, k, pos, inv, **kw)
    b4 = ela.qk_norm_rope_bwd(*f4, q, k, pos, inv, **kw)
    assert all(torch.equal(a, b) for a, b in zip(f3 + b3, f4 + b4))


@gpu
def test_offsets_past_32_bits(lib):
    """More than 2^31 elements in one tensor; rows at the end against the formulas."""
    H, N, d = 128, 131072 + 5, 128
    g = torch.Generator("cuda").manual_seed(9)
    q = torch.empty(1, N, H, d, dtype=torch.bfloat16, device="cuda")
    for a in range(0, N, 16384):
        q[:, a:a + 16384] = torch.randn(q[:, a:a + 16384].shape, generator=g, device="cuda").to(torch.bfloat16)
    q = q.transpose(1, 2)
    k = torch.zeros(1, 1, N, d, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    inv = 10000.0 ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64)
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    y, _ = ela.qk_norm_rope(q, k, pos, inv, q_weight=w)
    dx, _, _, _ = ela.qk_norm_rope_bwd(y, k, q, k, pos, inv, q_weight=w)
    for part in (slice(0, 4), slice(65534, 65540), slice(N - 4, N)):
        p = pos[part].view(1, 1, -1)
        check_forward(q[:, :, part], w, p, inv, (64,), EPS, False, y[:, :, part])
        t = ref.angles(p.cpu().numpy(), inv.cpu().numpy(), (64,))
        want, S, _, _ = ref.backward(f64(y[:, :, part]), f64(q[:, :, part]), f64(w), t, EPS, False)
        assert ref.excess(f64(dx[:, :, part]), want, S) <= 0


@gpu
def test_binding_refuses(lib):
    q, k, pos, inv, wq, wk, dqo, dko = inputs(2, 4, 2, 6, 64, 64, (32,), 100, seed=10)
    ok = dict(q_weight=wq, k_weight=wk)
    for bad in (dict(positions=pos.long()), dict(positions=pos[:, :, :5]), dict(inv_freq=inv.float()),
                dict(sections=(16, 15)), dict(q_weight=wq.float()), dict(k=k.float()), dict(q=q[:, :, :, :32]),
                dict(positions=pos.cpu()), dict(q_out=q.float()), dict(k_out=k[:, :1])):
        a = dict(q=q, k=k, positions=pos, inv_freq=inv, **ok)
        a.update(bad)
        with pytest.raises(ValueError):
            ela.qk_norm_rope(**a)
    with pytest.raises(ela.AttnError):
        ela.qk_norm_rope(q, k, pos, inv[:12].contiguous(), sections=(12,), **ok)
    with pytest.raises(ValueError):
        ela.qk_norm_rope_bwd(dqo, dko[:, :1], q, k, pos, inv, **ok)
    with pytest.raises(ela.AttnError):
        ela.qk_norm_rope_bwd(dqo, dko, q, k, pos, inv, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"), **ok)
