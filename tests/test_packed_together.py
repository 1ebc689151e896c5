"""The packed and paged calls run together as a program runs them (GPU).

Training: views of a fused projection's output -> query / key preparation -> packed attention -> its gradient, each
part written straight into its place in the projection's gradient -> the preparation's gradient.  Every stage is held to
its own bound on the tensors that the stage before wrote.

Serving: prompts by packed attention, their keys and values laid into a cache's pages; a tree of drafted tokens checked
by one call; then each path of the tree taken through packed attention as if its tokens had been decided.  The two ways to the
same rows read the same bf16 numbers, so both lie within their bounds of one 64-bit reference.
"""
import pytest
import torch

import exact_long_sequence_gb300 as ela
from packed_ref import bits, check, check_bwd, packed, packed_bwd, starts, tree
from test_qk_norm_rope import check_backward, check_forward

pytestmark = pytest.mark.gpu
EPS = 1e-6


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d,Hq,Hk", [(64, 4, 4), (128, 6, 2)])
def test_training_step(d, Hq, Hk):
    ql = [70, 1, 333, 128]
    qs = starts(ql)
    N = qs[-1]
    g = torch.Generator("cuda").manual_seed(d)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    qkv, do = rand(N, Hq + 2 * Hk, d), rand(N, Hq, d).transpose(0, 1)
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2))
    pos = torch.cat([torch.arange(n) for n in ql]).to(torch.int32).cuda()
    inv = 100.0 ** (-torch.arange(d // 2, dtype=torch.float64, device="cuda") / (d // 2))
    q, k, v = (x.transpose(0, 1) for x in qkv.split([Hq, Hk, Hk], 1))
    st = dev(qs)

    qr, kr = ela.qk_norm_rope(q[None], k[None], pos, inv, wq, wk, eps=EPS)
    o = torch.empty((N, Hq, d), dtype=torch.bfloat16, device="cuda").transpose(0, 1)  # token-major, as the next projection reads it
    o, lse = ela.attn_fwd_packed(qr[0], kr[0], v, st, causal=True, out=o)
    grad = torch.full_like(qkv, 7)
    gq, gk, gv = (x.transpose(0, 1) for x in grad.split([Hq, Hk, Hk], 1))
    dqr, dkr, dv = ela.attn_bwd_packed(qr[0], kr[0], v, o, lse, do, st, causal=True, dv=gv)
    _, _, dwq, dwk = ela.qk_norm_rope_bwd(dqr[None], dkr[None], q[None], k[None], pos, inv, wq, wk, eps=EPS, dq=gq[None], dk=gk[None])
    assert ela.last_device_error() == ela.ATTN_OK

    every, sec = pos.view(1, 1, N), (d // 2,)
    check_forward(q[None], wq, every, inv, sec, EPS, False, qr)
    check_forward(k[None], wk, every, inv, sec, EPS, False, kr)
    scale = ela.default_scale(d)
    check(o, lse, packed(qr[0], kr[0], v, qs, qs, True, scale))
    check_bwd((dqr, dkr, gv), *packed_bwd(qr[0], kr[0], v, o, lse, do, qs, qs, True, scale))
    check_backward(dqr[None], q[None], wq, every, inv, sec, EPS, False, gq[None], dwq)
    check_backward(dkr[None], k[None], wk, every, inv, sec, EPS, False, gk[None], dwk)


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
def test_prompts_then_a_tree_of_drafts(d, page):
    Hq, Hk, T = 8, 2, 6
    prompts = [37, 200, 64]
    R = len(prompts)
    g = torch.Generator("cuda").manual_seed(page)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    scale = ela.default_scale(d)
    # the prompts, packed
    qs = starts(prompts)
    q, k, v = rand(Hq, qs[-1], d), rand(Hk, qs[-1], d), rand(Hk, qs[-1], d)
    out, lse = ela.attn_fwd_packed(q, k, v, dev(qs), causal=True)
    check(out, lse, packed(q, k, v, qs, qs, True, scale))
    # their keys and values in pages, with room for the drafts
    need = [(n + T + page - 1) // page for n in prompts]
    ids = torch.randperm(sum(need), generator=g, device="cuda").tolist()
    table = torch.zeros((R, max(need)), dtype=torch.int32)
    kc, vc = (torch.zeros((sum(need), Hk, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for r in range(R):
        for i in range(need[r]):
            table[r, i] = ids.pop()

    def put(r, at, kk, vv):
        kc[table[r, at // page], :, at % page], vc[table[r, at // page], :, at % page] = kk, vv

    for r in range(R):
        for i in range(prompts[r]):
            put(r, i, k[:, qs[r] + i], v[:, qs[r] + i])
    parents = [-1, 0, 0, 1, 2, 2]
    paths = []
    for t, parent in enumerate(parents):
        paths.append((paths[parent] if parent >= 0 else []) + [t])
    seen = torch.zeros((R, T, T), dtype=torch.bool)
    for t in range(T):
        seen[:, t, paths[t]] = True
    qd, kd, vd = rand(R, Hq, T, d), rand(R, Hk, T, d), rand(R, Hk, T, d)
    for r in range(R):
        for t in range(T):
            put(r, prompts[r] + t, kd[r, :, t], vd[r, :, t])
    lens = [n + T for n in prompts]
    to, tl = ela.attn_fwd_tree(qd, kc, vc, table.cuda(), dev(lens), bits(seen).cuda())
    check(to, tl, tree(qd, kc, vc, table.cuda(), lens, seen.cuda(), scale))
    # each path as decided tokens behind the prompt, all of them in one packed call
    for t in range(T):
        path = paths[t]
        kp = torch.cat([torch.cat([k[:, qs[r]:qs[r + 1]], kd[r][:, path]], 1) for r in range(R)], 1)
        vp = torch.cat([torch.cat([v[:, qs[r]:qs[r + 1]], vd[r][:, path]], 1) for r in range(R)], 1)
        qp = torch.cat([qd[r][:, path] for r in range(R)], 1)
        qst, kst = starts([len(path)] * R), starts([n + len(path) for n in prompts])
        po, pl = ela.attn_fwd_packed(qp, kp, vp, dev(qst), dev(kst), causal=True)
        ref = packed(qp, kp, vp, qst, kst, True, scale)
        check(po, pl, ref)
        last = [e - 1 for e in qst[1:]]  # the draft itself, at the end of its path
        check(to[:, :, t].transpose(0, 1), tl[:, :, t].transpose(0, 1), tuple(x[:, last] for x in ref))
    assert ela.last_device_error() == ela.ATTN_OK
