"""The query / key preparation, the attention kernels and their gradients run together as a program
runs them, in training and in serving (GPU).

Bounds.  Within a chain every stage reads the bf16 tensors that the stage before wrote, so each
new operator is held to its own bound on exactly those tensors (qk_norm_rope_ref, test_prefix).  Over the
whole training chain the gradients are compared in the 2-norm with 64-bit autograd: there are ten
roundings to bf16 on the way (q, k, P twice, O, dO as drawn, dS twice, dQ / dK, the result), each off by at most 2^-8
of its value; scores of size |s| <= 6 pass a relative error on into P at most sixfold, in norm and with
signs as they fall by far less.  2^-8 * 10 is 2^-4.7: the bound is 2^-4.
"""
import math

import pytest
import torch

import exact_long_sequence_gb300 as ela

import qk_norm_rope_ref as ref
from test_prefix import check as check_prefix
from test_qk_norm_rope import check_backward, check_forward

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from exact_long_sequence_gb300 import _build

    _build.build()
    ela.load_library()


def weights(g, d):
    return [(1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2)]


@pytest.mark.parametrize("d,sections,interleaved", [(64, (32,), True), (128, (16, 24, 24), False)])
def test_training_step(d, sections, interleaved):
    """A fused projection's output -> norm and rotation -> causal attention, and back to its gradient."""
    B, N, H = 2, 300, 3
    g = torch.Generator("cuda").manual_seed(d)
    qkv = torch.randn(B, N, 3 * H, d, generator=g, device="cuda").to(torch.bfloat16)
    do = torch.randn(B, H, N, d, generator=g, device="cuda").to(torch.bfloat16)
    wq, wk = weights(g, d)
    pos = torch.stack([torch.arange(N, device="cuda") // (20 ** i) for i in range(len(sections))]).to(torch.int32)
    pos = pos[:, None]  # [axes, 1, N]: the same for both batches
    inv = 100.0 ** (-torch.arange(d // 2, dtype=torch.float64, device="cuda") / (d // 2))
    q, k, v = (qkv[:, :, i * H:(i + 1) * H].transpose(1, 2) for i in range(3))
    kw = dict(q_weight=wq, k_weight=wk, sections=sections, eps=EPS, interleaved=interleaved)

    qr, kr = ela.qk_norm_rope(q, k, pos, inv, **kw)
    vc = v.contiguous()
    o, lse = ela.attn_fwd(qr, kr, vc, causal=True)
    dqr, dkr, dv = ela.attn_bwd(qr, kr, vc, o, lse, do, causal=True)
    grad = torch.empty_like(qkv)  # the fused projection's gradient: the three parts in place
    dq, dk, dwq, dwk = ela.qk_norm_rope_bwd(dqr, dkr, q, k, pos, inv, dq=grad[:, :, :H].transpose(1, 2),
                                            dk=grad[:, :, H:2 * H].transpose(1, 2), **kw)
    grad[:, :, 2 * H:] = dv.transpose(1, 2)
    assert ela.last_device_error() == ela.ATTN_OK

    # each new stage on the tensors it was given
    every = pos.expand(len(sections), B, N)
    check_forward(q, wq, every, inv, sections, EPS, interleaved, qr)
    check_forward(k, wk, every, inv, sections, EPS, interleaved, kr)
    check_backward(dqr, q, wq, every, inv, sections, EPS, interleaved, dq, dwq)
    check_backward(dkr, k, wk, every, inv, sections, EPS, interleaved, dk, dwk)

    # the whole step against autograd in 64 bits
    x = qkv.double().requires_grad_()
    w = [t.double().requires_grad_() for t in (wq, wk)]
    t = torch.from_numpy(ref.angles(every.cpu().numpy(), inv.cpu().numpy(), sections)).cuda()
    a, b = (torch.from_numpy(i).cuda() for i in ref.pair_index(d // 2, interleaved))

    def ready(y, w):
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w
        out = torch.empty_like(y)
        out[..., a] = y[..., a] * t.cos() - y[..., b] * t.sin()
        out[..., b] = y[..., b] * t.cos() + y[..., a] * t.sin()
        return out

    q6, k6, v6 = (x[:, :, i * H:(i + 1) * H].transpose(1, 2) for i in range(3))
    z = ready(q6, w[0]) @ ready(k6, w[1]).transpose(2, 3) / math.sqrt(d)
    z = z.masked_fill(torch.ones(N, N, dtype=torch.bool, device="cuda").triu(1), -math.inf)
    want = torch.autograd.grad((torch.softmax(z, -1) @ v6 * do.double()).sum(), [x] + w)
    for got, ref6 in zip((grad, dwq, dwk), want):
        assert (got.double() - ref6).norm() <= 2.0 ** -4 * ref6.norm()


@pytest.mark.parametrize("T", [1, 3])
def test_serving_step(T):
    """A prompt is prepared into a cache's rows and attended once; then four requests continue it,
    each step preparing its new keys, appending them to its own cache and attending to both."""
    d, Hq, Hk, P, C, R = 128, 8, 2, 333, 40, 4
    g = torch.Generator("cuda").manual_seed(T)

    def draw(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    wq, wk = weights(g, d)
    inv = 10000.0 ** (-torch.arange(d // 2, dtype=torch.float64, device="cuda") / (d // 2))
    kw = dict(q_weight=wq, k_weight=wk, eps=EPS)
    # the prompt: its keys into the first rows of a larger cache
    cache_k, cache_v = (torch.full((Hk, 512, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, k, v = draw(1, Hq, P, d), draw(1, Hk, P, d), draw(Hk, P, d)
    cache_v[:, :P] = v
    qr, kr = ela.qk_norm_rope(q, k, torch.arange(P, dtype=torch.int32, device="cuda"), inv, k_out=cache_k[None, :, :P], **kw)
    o, lse = ela.attn_fwd(qr, kr.repeat_interleave(Hq // Hk, 1), v[None].repeat_interleave(Hq // Hk, 1), causal=True)
    assert ela.last_device_error() == ela.ATTN_OK and torch.isfinite(o).all()
    # the prompt's last token as a request without own keys sees the same keys
    last, last_lse = ela.attn_fwd_prefix(qr[:, :, -1:], cache_k[:, :P], cache_v[:, :P])
    check_prefix(dict(q=qr[:, :, -1:], k_prefix=cache_k[:, :P], v_prefix=cache_v[:, :P]), last, last_lse)
    assert (last_lse[0, :, 0] - lse[0, :, -1]).abs().max() <= 2.0 ** -12 * (1 + lse.abs().max())

    own_k, own_v = (torch.full((R, Hk, C, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    out, ol = torch.empty(R, Hq, T, d, dtype=torch.bfloat16, device="cuda"), torch.empty(R, Hq, T, device="cuda")
    for step in range(4):
        grow = torch.full((R,), T, dtype=torch.int32, device="cuda")
        if step == 2:
            lens[1] = -lens[1]  # request 1 has ended: padding from here on
            grow[1] = 0
        before = out.clone()
        at = lens.clamp(min=0)
        q, k, v = draw(R, Hq, T, d), draw(R, Hk, T, d), draw(R, Hk, T, d)
        pos = (P + at[:, None] + torch.arange(T, device="cuda")).to(torch.int32)
        qr, kr = ela.qk_norm_rope(q, k, pos, inv, **kw)
        rows = (at[:, None] + torch.arange(T, device="cuda")).long()
        for r in range(R):
            own_k[r, :, rows[r]], own_v[r, :, rows[r]] = kr[r], v[r]
        lens += grow
        ela.attn_fwd_prefix(qr, cache_k[:, :P], cache_v[:, :P], own_k, own_v, lens, out=out, lse=ol)
        s = dict(q=qr, k_prefix=cache_k[:, :P], v_prefix=cache_v[:, :P], k_own=own_k, v_own=own_v, own_lens=lens)
        check_prefix(s, out, ol)
        if step >= 2:
            assert torch.equal(out[1], before[1])
