"""The query / key preparation and its gradient in 64 bits, written from the formulas, with the
bounds that the GPU results are held to.

Bounds.  The kernels compute in fp32 and round each output once to bf16, which is off by at most
2^-8 of the value.  Before that rounding an element is a sum of at most a few products of
magnitudes summing to S (both members of its pair, and in the gradient the mean's term); each
factor (norm, sine, cosine, weight product, mean over at most 128 elements summed pairwise or in
chains of 16) carries a relative error below 2^-20, so the fp32 value is off by at most 2^-18 S.
With e = 2^-18 S the rounded value is off by at most e + 2^-8 (|ref| + e).  A weight gradient is an fp32
sum of n terms, off by at most (2^-18 + n 2^-24) of the sum of their magnitudes.
"""
import numpy as np


def pair_index(pairs, interleaved):
    i = np.arange(pairs)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)


def angles(positions, inv_freq, sections):
    """positions [A, B, N] ints -> radians [B, 1, N, pairs].  The product is taken modulo a turn in
    extended integers' place: float64 holds it to 2^-53 of the angle, checked by the caller's choice of positions."""
    axis = np.repeat(np.arange(len(sections)), sections)
    p = np.asarray(positions, dtype=np.float64)[axis]  # [pairs, B, N]
    return (np.moveaxis(p, 0, -1) * np.asarray(inv_freq, dtype=np.float64))[:, None]


def turn(x, t, interleaved, sign=1):
    a, b = pair_index(t.shape[-1], interleaved)
    y = x.copy()
    c, s = np.cos(t), np.sin(t) * sign
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def spread(x, pairs, interleaved):
    """|x| with each rotated element replaced by its pair's |a| + |b|."""
    a, b = pair_index(pairs, interleaved)
    y = np.abs(x)
    s = y[..., a] + y[..., b]
    y[..., a] = s
    y[..., b] = s
    return y


def forward(x, w, t, eps, interleaved):
    """(output, the magnitude S of the bound); x float64 [B, H, N, d]."""
    y = x
    if w is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return turn(y, t, interleaved), spread(y, t.shape[-1], interleaved)


def backward(dy, x, w, t, eps, interleaved):
    """(dx, its S, dw, the sum of the magnitudes of dw's terms)."""
    u = turn(dy, t, interleaved, -1)
    U = spread(dy, t.shape[-1], interleaved)
    if w is None:
        return u, U, None, None
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    h = x * r
    dx = r * (u * w - h * (u * w * h).mean(-1, keepdims=True))
    S = r * (U * np.abs(w) + np.abs(h) * (U * np.abs(w * h)).mean(-1, keepdims=True))
    return dx, S, (u * h).sum((0, 1, 2)), (U * np.abs(h)).sum((0, 1, 2))


def excess(got, ref, S):
    """How far a bf16 result lies outside its bound (<= 0: inside)."""
    e = 2.0 ** -18 * S
    return float((np.abs(got - ref) - (e + 2.0 ** -8 * (np.abs(ref) + e) + 1e-38)).max())
