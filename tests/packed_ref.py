"""Plain 64-bit attention over packed sequences and paged caches, and the error bounds of the kernels against it."""
import math

import torch


def attention(q, k, v, seen, scale):
    """q [H, n, d], k, v [H, m, d] doubles, seen [n, m] truth values: O, LSE and sum_j p_j |v_j| per element."""
    s = torch.matmul(q, k.transpose(-1, -2)) * scale
    s = s.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1) if s.shape[-1] else torch.full(s.shape[:-1], -math.inf, dtype=s.dtype, device=s.device)
    p = torch.where(seen, torch.exp(s - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[..., None]),
                    torch.zeros_like(s))
    return torch.matmul(p, v), lse, torch.matmul(p, v.abs())


def packed(q, k, v, q_starts, k_starts, causal, scale):
    """The definition, sequence by sequence; rows in no sequence are NaN in all three results."""
    Hq, Nq, d = q.shape
    G = Hq // k.shape[0]
    nan = lambda *s: torch.full(s, math.nan, dtype=torch.float64, device=q.device)  # noqa: E731
    o, lse, a = nan(Hq, Nq, d), nan(Hq, Nq), nan(Hq, Nq, d)
    for (q0, q1), (k0, k1) in zip(zip(q_starts, q_starts[1:]), zip(k_starts, k_starts[1:])):
        n, m = max(0, q1 - q0), max(0, k1 - k0)
        if n == 0:
            continue
        i = torch.arange(n, device=q.device)[:, None]
        seen = torch.arange(m, device=q.device) <= (i + m - n if causal else m + 0 * i)
        kk, vv = (x[:, k0:k0 + m].double().repeat_interleave(G, 0) for x in (k, v))
        o[:, q0:q1], lse[:, q0:q1], a[:, q0:q1] = attention(q[:, q0:q1].double(), kk, vv, seen, scale)
    return o, lse, a


def tree(q, kc, vc, table, lens, seen_new, scale):
    """seen_new: [R, T, T] truth values; requests of negative length are NaN."""
    R, Hq, T, d = q.shape
    Hk, page = kc.shape[1], kc.shape[2]
    G = Hq // Hk
    nan = lambda *s: torch.full(s, math.nan, dtype=torch.float64, device=q.device)  # noqa: E731
    o, lse, a = nan(R, Hq, T, d), nan(R, Hq, T), nan(R, Hq, T, d)
    for r, n in enumerate(lens):
        if n < 0:
            continue
        n = min(n, table.shape[1] * page)
        ids = table[r, : (n + page - 1) // page].long()
        kk, vv = (x[ids].double().transpose(0, 1).reshape(Hk, -1, d)[:, :n].repeat_interleave(G, 0) for x in (kc, vc))
        at = torch.arange(n, device=q.device) - (n - T)
        seen = torch.where(at < 0, True, seen_new[r][:, at.clamp(min=0)])
        o[r], lse[r], a[r] = attention(q[r].double(), kk, vv, seen, scale)
    return o, lse, a


def check(o, lse, ref):
    """Elementwise bounds.  P is rounded to bf16 (half a step: 2^-8 of each term), O once more; scores are fp32 sums of
    exact products, whose rounding moves a term by at most 2^-12 at these sizes (d 2^-24 of the terms' sum), and the
    sums of the terms and the merges of pieces by less.  The log-sum-exp moves as much as a term."""
    ro, rl, ra = ref
    live = ~torch.isnan(rl)
    err = (o.double() - ro).abs()
    tol = 2.0 ** -8 * (ra + ro.abs()) + 2.0 ** -11 * ra + 1e-30
    assert bool((err <= tol)[live].all()), f"O off by {(err / tol)[live].max().item():.3f} of its bound"
    none = live & (rl == -math.inf)
    assert bool((lse[none] == -math.inf).all()) and bool((o[none] == 0).all())
    some = live & ~none
    gap = (lse.double() - rl).abs()[some]
    assert gap.numel() == 0 or gap.max().item() <= 2.0 ** -12 + 1e-6 * rl[some].abs().max().item(), gap.max().item()


def bits(seen):
    """[R, T, T] truth values as the rows of 32-bit words that attn_fwd_tree takes."""
    R, T, _ = seen.shape
    w = (T + 31) // 32
    x = torch.zeros((R, T, w * 32), dtype=torch.int64)
    x[..., :T] = seen.cpu().long()
    x = (x.view(R, T, w, 32) << torch.arange(32)).sum(-1)
    return torch.where(x >= 1 << 31, x - (1 << 32), x).to(torch.int32)


def starts(lens, first=0):
    out = [first]
    for n in lens:
        out.append(out[-1] + n)
    return out


def packed_bwd(q, k, v, o, lse, do, q_starts, k_starts, causal, scale):
    """The gradients' formulas for the forward's o and lse, sequence by sequence, and a bound of the kernel's error:
    (dq, dk, dv), (tq, tk, tv); rows in no sequence are NaN.

    P is rounded to bf16 (2^-8 of it), dS again (2^-8), and each result once more (2^-8); P moves with the scores and the
    LSE as in the forward (2^-12), the difference dP - D by the rounding of fp32 sums (at most 2^-16 of their terms' sum),
    and the sums over rows and keys by at most 2^-10 of their terms' sum (up to 2^13 of them in fp32)."""
    Hq, Nq, d = q.shape
    Hk = k.shape[0]
    G = Hq // Hk
    nan = lambda t: torch.full(t.shape, math.nan, dtype=torch.float64, device=q.device)  # noqa: E731
    dq, dk, dv, tq, tk, tv = nan(q), nan(k), nan(v), nan(q), nan(k), nan(v)
    step = 2.0 ** -8
    for (q0, q1), (k0, k1) in zip(zip(q_starts, q_starts[1:]), zip(k_starts, k_starts[1:])):
        n, m = max(0, q1 - q0), max(0, k1 - k0)
        qs, ks = slice(q0, q0 + n), slice(k0, k0 + m)
        i = torch.arange(n, device=q.device)[:, None]
        seen = torch.arange(m, device=q.device) <= (i + m - n if causal else m + 0 * i)
        for x in (dk, dv, tk, tv):
            x[:, ks] = 0
        for h in range(Hq):
            Q, K, V, O, g = (x.double() for x in (q[h, qs], k[h // G, ks], v[h // G, ks], o[h, qs], do[h, qs]))
            p = torch.where(seen, torch.exp(Q @ K.T * scale - lse[h, qs].double()[:, None]), 0.0)
            D = (g * O).sum(-1, keepdim=True)
            ds = p * (g @ V.T - D) * scale
            e = ds.abs() * (2 * step + 2.0 ** -9) + p * abs(scale) * 2.0 ** -16 * (g.abs() @ V.abs().T + (g * O).abs().sum(-1, keepdim=True))
            dq[h, qs] = ds @ K
            tq[h, qs] = e @ K.abs() + step * dq[h, qs].abs()
            dk[h // G, ks] += ds.T @ Q
            tk[h // G, ks] += e.T @ Q.abs()
            dv[h // G, ks] += p.T @ g
            tv[h // G, ks] += (p * (step + 2.0 ** -9)).T @ g.abs()
    return (dq, dk, dv), (tq, tk + step * dk.abs(), tv + step * dv.abs())


def check_bwd(got, ref, tol):
    for name, x, r, t in zip(("dq", "dk", "dv"), got, ref, tol):
        live = ~torch.isnan(r)
        err = (x.double() - r).abs()
        # (a gradient that is the difference of equal sums may be far below them: 2^-133 is bf16's smallest number)
        assert bool((err <= t + 2.0 ** -133)[live].all()), f"{name} off by {(err / (t + 2.0 ** -133))[live].max().item():.3f} of its bound"
