"""Attention of a batch over a shared prefix and each request's own keys: refusals on the CPU, parity
with the definition in 64 bits on the GPU.

Bounds.  Scores are fp32 sums of d exact bf16 products: off by at most ds = scale * sum_c |q_c k_c| * d * 2^-23
(an error of a step at every addition).  A weight p is off by 2 ds relatively (its exponent and the
maximum's), by 2^-20 for exp2, and its bf16 rounding by 2^-8, so with A = sum_j p_j |v_j| / l
    |dO| <= (2 ds + 2^-8 + 2^-16) A + 2^-8 (|O| + that)     (the second rounding: O itself)
where 2^-16 covers the fp32 sums over the keys and the merging of the pieces (relative to A).
    |dLSE| <= ds + 2^-18 (1 + |LSE|).
"""
import ctypes
import math

import pytest
import torch

import exact_long_sequence_gb300 as ela
from exact_long_sequence_gb300 import _build

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ela.load_library()


def cdll_call(lib, **over):
    a = dict(Q=0x1000, qs=None, Kp=0x2000, kps=None, Vp=0x3000, vps=None, Ko=0x4000, kos=None, Vo=0x5000, vos=None,
             lens=0x6000, O=0x7000, os=None, LSE=0x8000, R=3, Hq=8, Hk=2, T=1, P=100, C=50, d=64, scale=0.125,
             ws=0x9000, wsb=1 << 40)
    a.update(over)
    for k, n in (("qs", 3), ("kps", 2), ("vps", 2), ("kos", 3), ("vos", 3), ("os", 3)):
        a[k] = (ctypes.c_int64 * n)(*a[k]) if a[k] is not None else None
    return lib.attn_fwd_prefix(*[a[k] for k in ("Q", "qs", "Kp", "kps", "Vp", "vps", "Ko", "kos", "Vo", "vos", "lens",
                                                "O", "os", "LSE", "R", "Hq", "Hk", "T", "P", "C", "d", "scale", "ws",
                                                "wsb")], None)


@pytest.mark.parametrize("over,status", [
    (dict(Q=None), 1), (dict(O=None), 1), (dict(LSE=None), 1), (dict(Kp=None), 1), (dict(Vo=None), 1),
    (dict(lens=None), 1), (dict(ws=None), 1), (dict(R=0), 1), (dict(T=0), 1), (dict(Hk=0), 1), (dict(P=-1), 1),
    (dict(C=-1), 1), (dict(P=0, C=0), 1), (dict(Hk=3), 1), (dict(R=1 << 20, Hq=1 << 10, T=4), 1),
    (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1), (dict(d=96), 2), (dict(Q=0x1004), 3),
    (dict(Vp=0x3008), 3), (dict(Ko=0x4002), 3), (dict(O=0x7008), 3), (dict(LSE=0x8002), 3), (dict(lens=0x6001), 3),
    (dict(ws=0x9008), 3), (dict(qs=(512, 68, 64)), 3), (dict(kps=(6400, 0)), 1), (dict(vos=(6400, -64, 64)), 1),
    (dict(kps=(1 << 39, 64)), 1), (dict(R=1 << 20, C=1 << 14), 1), (dict(qs=(1 << 38, 64, 64)), 1),
])
def test_refusals(lib, over, status):
    assert cdll_call(lib, **over) == status


def test_sizes_of_invalid_shapes(lib):
    for bad in ((0, 8, 2, 1, 10, 10, 64), (1, 8, 3, 1, 10, 10, 64), (1, 8, 2, 1, 0, 0, 64), (1, 8, 2, 1, 10, 10, 80)):
        assert lib.attn_fwd_prefix_workspace_bytes(*bad) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_valid_calls_without_gpu_report_no_device(lib):
    none = (ela.ATTN_ERR_NO_DEVICE, ela.ATTN_ERR_CUDA)
    assert cdll_call(lib) in none
    assert cdll_call(lib, P=0, Kp=None, Vp=None) in none and cdll_call(lib, C=0, Ko=None, Vo=None, lens=None) in none
    assert cdll_call(lib, Hk=1, Hq=1, kps=(0, 64), qs=(64, 3, 64)) in none  # strides of axes of one are not looked at


def test_binding_refuses_on_the_host():
    q = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ela.attn_fwd_prefix(q, q[0], q[0])


# ------------------------------------------------------------------ GPU
def make(R, Hq, Hk, T, d, P, C, lens, seed, token_major=False, spiky=False, garbage=True):
    g = torch.Generator("cuda").manual_seed(seed)

    def draw(*shape):
        x = torch.randn(shape, generator=g, device="cuda")
        if spiky:
            x = x * torch.where(torch.rand(shape, generator=g, device="cuda") < 0.01, 10.0, 1.0)
        return x.to(torch.bfloat16)

    s = dict(q=draw(R, Hq, T, d))
    if P:
        s["k_prefix"], s["v_prefix"] = draw(Hk, P, d), draw(Hk, P, d)
        if token_major:
            s["k_prefix"], s["v_prefix"] = (s[k].transpose(0, 1).contiguous().transpose(0, 1) for k in ("k_prefix", "v_prefix"))
    if C:
        k, v = draw(R, Hk, C, d), draw(R, Hk, C, d)
        if token_major:
            k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))
        for r, n in enumerate(lens):
            if garbage:  # what lies past a request's keys is not read as numbers
                k[r, :, max(0, min(n, C)):] = float("nan")
                v[r, :, max(0, min(n, C)):] = float("inf") if r % 2 else float("nan")
        s["k_own"], s["v_own"] = k, v
        s["own_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return s


def check(s, out, lse, scale=None, requests=None):
    """Against the definition, request by request, with the bounds above."""
    q = s["q"]
    R, Hq, T, d = q.shape
    scale = 1 / math.sqrt(d) if scale is None else scale
    kp, vp = s.get("k_prefix"), s.get("v_prefix")
    ko = s.get("k_own")
    Hk = kp.shape[0] if kp is not None else ko.shape[1]
    lens = s["own_lens"].tolist() if ko is not None else [0] * R
    C = ko.shape[2] if ko is not None else 0
    assert ela.last_device_error() == ela.ATTN_OK
    for r in range(R) if requests is None else requests:
        if lens[r] < 0:
            continue
        n = min(lens[r], C)
        K = torch.cat([x for x in (kp, ko[r, :, :n] if ko is not None else None) if x is not None], 1).double()
        V = torch.cat([x for x in (vp, s["v_own"][r, :, :n] if ko is not None else None) if x is not None], 1).double()
        P = K.shape[1] - n
        Q = q[r].double().view(Hk, Hq // Hk, T, d)
        z = torch.einsum("hgtd,hkd->hgtk", Q, K) * scale
        ds = torch.einsum("hgtd,hkd->hgtk", Q.abs(), K.abs()).amax(-1) if K.shape[1] else torch.zeros_like(z).sum(-1)
        ds = ds * abs(scale) * d * 2.0 ** -23
        last = P + n - (T - 1) + torch.arange(T, device="cuda").clamp(max=T - 1)
        seen = (torch.arange(P + n, device="cuda") < P) | (torch.arange(P + n, device="cuda") < last[:, None])
        z = z.masked_fill(~seen, -math.inf)
        want_l = torch.logsumexp(z, -1) if z.shape[-1] else torch.full_like(ds, -math.inf)
        p = torch.exp(z - torch.where(want_l.isinf(), 0.0, want_l)[..., None])
        want = torch.einsum("hgtk,hkd->hgtd", p, V)
        A = torch.einsum("hgtk,hkd->hgtd", p, V.abs())
        got, got_l = out[r].double().view_as(want), lse[r].double().view_as(want_l)
        e = (2 * ds[..., None] + 2.0 ** -8 + 2.0 ** -16) * A
        assert torch.isfinite(got).all()
        bad = (got - want).abs() - (e + 2.0 ** -8 * (want.abs() + e) + 1e-30)
        assert (bad <= 0).all(), f"request {r}: O outside its bound by {bad.max().item():.3e}"
        none = want_l == -math.inf
        assert torch.equal(got_l == -math.inf, none)
        assert (got[none] == 0).all()
        bad = ((got_l - want_l).abs() - (ds + 2.0 ** -18 * (1 + want_l.abs())))[~none]
        assert (bad <= 0).all(), f"request {r}: LSE outside its bound by {bad.max().item():.3e}"


# R, Hq, Hk, T, d, P, C, own lengths, token-major caches
SHAPES = [
    (1, 1, 1, 1, 64, 1, 0, [], False),
    (1, 1, 1, 1, 128, 0, 1, [1], False),
    (2, 4, 2, 1, 128, 100, 40, [17, 40], False),
    (3, 8, 8, 1, 64, 128, 33, [0, 1, 33], True),
    (5, 8, 1, 1, 128, 129, 16, [16, 0, 3, 15, 1], True),
    (4, 32, 4, 1, 128, 1000, 300, [300, 129, 128, 127], False),
    (6, 16, 2, 1, 64, 4097, 500, [500, 31, 32, 33, 64, 65], False),
    (17, 8, 1, 1, 128, 777, 20, list(range(4, 21)), False),         # 136 rows: two query tiles, the second short
    (40, 8, 1, 1, 64, 515, 260, [(7 * i) % 261 for i in range(40)], True),  # 320 rows: two blocks
    (3, 4, 2, 5, 128, 300, 200, [5, 200, 77], False),               # several new tokens
    (2, 8, 2, 4, 64, 0, 130, [4, 130], True),
    (2, 2, 1, 3, 128, 50, 9, [1, 2], False),                        # fewer own keys than new tokens
    (2, 8, 1, 33, 128, 260, 400, [33, 400], False),                 # 264 rows of a request: two own blocks
    (50, 12, 2, 3, 128, 700, 40, [(3 * i) % 41 for i in range(50)], True),  # 18 rows a request: tiles of 126 rows
    (5, 20, 2, 3, 128, 100, 1100, [1100, 0, 2, 700, 129], False),   # 30 rows, caches too long for row blocks
    (5, 20, 2, 3, 64, 100, 700, [700, 0, 2, 16, 129], True),        # 30 rows in blocks of 15
    (5, 20, 2, 3, 64, 0, 700, [700, 0, 2, 16, 129], True),          # ... without a prefix: the own-keys kernel
    (3, 44, 4, 4, 128, 0, 64, [64, 17, 5], False),
    (60, 21, 3, 3, 128, 100, 90, [(7 * i) % 91 for i in range(60)], True),  # 180 sequences beside a prefix
    (200, 4, 1, 1, 64, 300, 50, [(3 * i) % 51 for i in range(200)], False),
    (3, 44, 4, 4, 128, 60, 64, [64, 17, 5], False),                 # 44 rows in blocks of 16, the last of 12
    (9, 33, 1, 2, 64, 300, 20, [20] * 9, False),                    # 66 rows a request: one a tile
    (3, 128, 1, 1, 128, 300, 33, [33, 0, 7], False),                # 128 rows a request: one a tile
    (3, 16, 2, 17, 64, 200, 50, [50, 17, 20], False),               # 136 rows a request: rows fetched one by one
    (1, 64, 1, 1, 128, 0, 5000, [4999], False),                     # a long own part alone, cut over many CTAs
    (1, 8, 8, 1, 64, 40000, 0, [], False),
    (3, 3, 3, 1, 128, 200, 64, [70, 64, 1 << 30], False),           # lengths past the capacity
    (130, 4, 4, 1, 128, 0, 70, [(11 * i) % 71 for i in range(130)], False),
]


@gpu
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s[:7])))
def test_parity(lib, shape):
    R, Hq, Hk, T, d, P, C, lens, major = shape
    s = make(R, Hq, Hk, T, d, P, C, lens, seed=R + P + C, token_major=major)
    out = torch.full((R, Hq, T, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((R, Hq, T), float("nan"), device="cuda")
    ela.attn_fwd_prefix(**s, out=out, lse=lse)
    check(s, out, lse)


@gpu
@pytest.mark.parametrize("lens", ["zero", "short", "full", "one", "any"])
@pytest.mark.parametrize("R,Hq,Hk,d,P,C", [(40, 16, 8, 64, 16384, 500), (256, 32, 8, 128, 5000, 100), (120, 3, 3, 128, 20001, 400)])
def test_prefix_beside_the_own_keys(lib, R, Hq, Hk, d, P, C, lens):
    """Shapes whose prefix starts beside the own-keys kernel, on stretches that follow from the lengths."""
    n = {"zero": lambda i: 0, "short": lambda i: 1 + i % 7, "full": lambda i: C, "one": lambda i: C if i == 3 else 0,
         "any": lambda i: (i * 37) % (C + 1) - (i % 11 == 0)}[lens]
    s = make(R, Hq, Hk, 1, d, P, C, [n(i) for i in range(R)], seed=R)
    out = torch.full((R, Hq, 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((R, Hq, 1), 7.0, device="cuda")
    ela.attn_fwd_prefix(**s, out=out, lse=lse)
    check(s, out, lse, requests=range(0, R, 5))
    pad = s["own_lens"] < 0
    assert (out[pad] == 7.0).all() and torch.isfinite(out).all() and torch.isfinite(lse).all()


@gpu
def test_rows_without_any_key(lib):
    """No prefix and no own keys for a request, or for its first tokens: O = 0, LSE = -inf."""
    s = make(4, 4, 2, 3, 64, 0, 50, [0, 1, 2, 50], seed=1)
    out, lse = ela.attn_fwd_prefix(**s)
    check(s, out, lse)
    assert (lse[0] == -math.inf).all() and (lse[1, :, :2] == -math.inf).all() and torch.isfinite(lse[3]).all()


@gpu
def test_padding_requests_are_left_as_they_were(lib):
    s = make(6, 8, 2, 2, 128, 200, 90, [90, -1, 5, -7, 0, 33], seed=2)
    out = torch.full((6, 8, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((6, 8, 2), 7.0, device="cuda")
    ela.attn_fwd_prefix(**s, out=out, lse=lse)
    check(s, out, lse)
    for r in (1, 3):
        assert (out[r] == 7.0).all() and (lse[r] == 7.0).all()


@gpu
def test_padding_without_own_keys(lib):
    s = make(4, 4, 2, 1, 64, 150, 0, [], seed=13)
    out = torch.full((4, 4, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 4, 1), 7.0, device="cuda")
    ela.attn_fwd_prefix(**s, own_lens=torch.tensor([0, -1, 5, -1], dtype=torch.int32, device="cuda"), out=out, lse=lse)
    for r in (1, 3):
        assert (out[r] == 7.0).all() and (lse[r] == 7.0).all()
    keep = [0, 2]
    check(dict(s, q=s["q"][keep]), out[keep], lse[keep])
    # an empty cache is the same as none
    empty = torch.empty(4, 2, 0, 64, dtype=torch.bfloat16, device="cuda")
    a = ela.attn_fwd_prefix(**s, k_own=empty, v_own=empty, own_lens=torch.zeros(4, dtype=torch.int32, device="cuda"))
    b = ela.attn_fwd_prefix(**s)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@gpu
@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0, 1e-30])
def test_any_finite_scale(lib, scale):
    s = make(3, 8, 2, 1, 128, 600, 150, [150, 20, 0], seed=3)
    out, lse = ela.attn_fwd_prefix(**s, scale=scale)
    check(s, out, lse, scale=scale)


@gpu
def test_rare_large_entries_move_the_reference_maximum(lib):
    s = make(20, 16, 2, 1, 128, 3000, 400, [20 * i for i in range(20)], seed=4, spiky=True)
    out, lse = ela.attn_fwd_prefix(**s, scale=1.0)
    check(s, out, lse, scale=1.0)


@gpu
def test_agrees_with_the_plain_forward(lib):
    """One request without a prefix, T = N new tokens: causal self-attention, as attn_fwd computes it."""
    N = 200
    g = torch.Generator("cuda").manual_seed(5)
    q, k, v = (torch.randn(1, 2, N, 64, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    o, l = ela.attn_fwd(q, k, v, causal=True)
    out, lse = ela.attn_fwd_prefix(q, None, None, k, v, torch.tensor([N], dtype=torch.int32, device="cuda"))
    # both round P and O to bf16: |O| <= max |v|
    assert (out.float() - o.float()).abs().max() <= 4 * 2.0 ** -8 * v.float().abs().max()
    assert (lse - l).abs().max() <= 2.0 ** -14


@gpu
def test_views_workspace_and_outputs_stay_inside_their_buffers(lib):
    R, Hq, Hk, T, d, P, C = 5, 8, 2, 2, 128, 333, 70
    s = make(R, Hq, Hk, T, d, P, C, [70, 2, 33, 8, 64], seed=6)
    want = ela.attn_fwd_prefix(**s)
    # the prefix as the first rows of a larger cache, the own caches inside a block of both, q and out token-major
    big = torch.full((Hk, P + 50, 2 * d), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[:, :P, :d], big[:, :P, d:] = s["k_prefix"], s["v_prefix"]
    kv = torch.full((R, C + 9, Hk, 2, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    kv[:, :C, :, 0], kv[:, :C, :, 1] = s["k_own"].transpose(1, 2), s["v_own"].transpose(1, 2)
    q = s["q"].transpose(1, 2).contiguous().transpose(1, 2)
    obuf = torch.full((R, T, Hq + 1, d), 3.0, dtype=torch.bfloat16, device="cuda")
    need = ela.prefix_workspace_bytes(R, Hq, Hk, T, P, C, d)
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    out, lse = ela.attn_fwd_prefix(q, big[:, :P, :d], big[:, :P, d:], kv[:, :C, :, 0].transpose(1, 2),
                                   kv[:, :C, :, 1].transpose(1, 2), s["own_lens"], out=obuf[:, :, :Hq].transpose(1, 2),
                                   workspace=ws[:need])
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert (obuf[:, :, Hq] == 3.0).all() and (ws[need:] == 0x5A).all()
    with pytest.raises(ela.AttnError):
        ela.attn_fwd_prefix(**s, workspace=ws[:need - 16])


@gpu
@pytest.mark.parametrize("R", [30, 100])  # own keys as items of the prefix kernel, and in a kernel of their own
def test_streams_graphs_and_repeated_calls(lib, R):
    Hq, Hk, T, d, P, C = 8, 2, 1, 128, 2000, 300
    lens = [(13 * i) % 301 for i in range(R)]
    s = make(R, Hq, Hk, T, d, P, C, [C] * R, seed=7)
    s["own_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    a = ela.attn_fwd_prefix(**s)
    b = ela.attn_fwd_prefix(**s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = ela.attn_fwd_prefix(**s, stream=side)
    side.synchronize()
    for x in (b, c):
        assert torch.equal(a[0], x[0]) and torch.equal(a[1], x[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = ela.attn_fwd_prefix(**s)
    # other lengths and queries in the same buffers (the caches hold numbers up to their capacity)
    for shift in (0, 1, 100):
        s["own_lens"].copy_(torch.tensor([(n + shift) % 301 for n in lens], dtype=torch.int32))
        s["q"].copy_(s["q"].roll(shift, 0))
        graph.replay()
        want = ela.attn_fwd_prefix(**s)
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])
        check(s, *g)


@gpu
def test_two_calls_at_once_with_a_workspace_each(lib):
    s = make(100, 8, 2, 1, 128, 3000, 200, [2 * i for i in range(100)], seed=8)
    t = make(16, 8, 2, 1, 128, 3000, 200, [200 - 12 * i for i in range(16)], seed=9)
    want = ela.attn_fwd_prefix(**s), ela.attn_fwd_prefix(**t)
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        a = ela.attn_fwd_prefix(**s, stream=one)
        b = ela.attn_fwd_prefix(**t, stream=two)
        torch.cuda.synchronize()
        for got, w in ((a, want[0]), (b, want[1])):
            assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])


@gpu
@pytest.mark.parametrize("P", [300, 0])
def test_a_nonfinite_request_stays_alone(lib, P):
    s = make(5, 8, 2, 1, 64, P, 60, [60, 60, 30, 7, 60], seed=10)
    clean = ela.attn_fwd_prefix(**s)
    s["k_own"][1, 0, 3, 5] = float("nan")
    s["v_own"][3, 1, 2, 9] = float("inf")
    out, lse = ela.attn_fwd_prefix(**s)
    assert out[1, :4].isnan().all() and lse[1, :4].isnan().all()
    assert (out[3, 4:, 0, 9] == float("inf")).all()
    same = torch.ones(5, 8, dtype=torch.bool)
    same[1, :4] = same[3, 4:] = False
    assert torch.equal(out.cpu()[same], clean[0].cpu()[same]) and torch.equal(lse.cpu()[same], clean[1].cpu()[same])


@gpu
def test_offsets_past_32_bits(lib):
    """A prefix and own caches of more than 2^31 elements each."""
    Hk, d, P = 8, 128, 2_100_000
    g = torch.Generator("cuda").manual_seed(11)
    kp, vp = (torch.empty(Hk, P, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for x in (kp, vp):
        for h in range(Hk):
            x[h] = torch.randn(P, d, generator=g, device="cuda").to(torch.bfloat16)
    q = (torch.randn(2, Hk, 1, d, generator=g, device="cuda")).to(torch.bfloat16)
    out, lse = ela.attn_fwd_prefix(q, kp, vp)
    assert ela.last_device_error() == ela.ATTN_OK
    for h in (0, Hk - 1):
        check(dict(q=q[:, h:h + 1], k_prefix=kp[h:h + 1], v_prefix=vp[h:h + 1]), out[:, h:h + 1], lse[:, h:h + 1])
    C = P  # the same memory as own caches of two requests with four heads each
    ko, vo = kp.view(2, 4, C, d), vp.view(2, 4, C, d)
    for lens in ([5, C], [C, 100]):
        s = dict(q=q[:, :4].contiguous(), k_own=ko, v_own=vo, own_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        out, lse = ela.attn_fwd_prefix(**s)
        for r in (0, 1):
            n = lens[r]
            one = dict(q=s["q"][r:r + 1, 3:], k_prefix=ko[r, 3:, :n], v_prefix=vo[r, 3:, :n])
            check(one, out[r:r + 1, 3:], lse[r:r + 1, 3:])


@gpu
def test_binding_refuses(lib):
    s = make(3, 8, 2, 1, 64, 100, 20, [1, 2, 3], seed=12)
    for bad in (dict(q=s["q"].float()), dict(q=s["q"][..., :32]), dict(v_prefix=s["v_prefix"][:1]), dict(v_prefix=None),
                dict(k_own=s["k_own"][:2]), dict(own_lens=s["own_lens"].long()), dict(own_lens=None),
                dict(own_lens=s["own_lens"].cpu()), dict(k_prefix=None, v_prefix=None, k_own=None, v_own=None),
                dict(out=s["q"].float()), dict(lse=torch.empty(3, 8, device="cuda")),
                dict(workspace=torch.empty(1 << 24, device="cuda"))):
        with pytest.raises(ValueError):
            ela.attn_fwd_prefix(**{**s, **bad})
    with pytest.raises(ela.AttnError):
        ela.attn_fwd_prefix(s["q"][:, :7], s["k_prefix"], s["v_prefix"])  # heads that do not divide
