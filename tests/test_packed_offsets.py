"""Offsets that lie outside the tensors or fall (a sequence whose end is before its start is empty), in both directions.

A batch padded to a fixed number of sequences has zeros or -1 behind the last one; every token that a sequence has gets its
gradient, and rows of tokens that are in none stay as they were.
"""
import math

import pytest
import torch

import exact_long_sequence_gb300 as ela
from packed_ref import check, check_bwd, packed, packed_bwd

pytestmark = pytest.mark.gpu

STARTS = [
    [0, 60, 100, 0],                          # padded with zeros
    [0, 60, 100] + [0] * 14,
    [0, 13, 97, -1, -1, -1, -1, -1],
    [0] + [7 * i for i in range(1, 12)] + [0] * 90,
    [-5, 40, 90, 2000, 7, 3, -1],             # clipped at both ends
    [1 << 30, 50, 20, 61],                    # falls before the only sequence
    [90, 95, 30, 0, 20, 10, 0],               # sequences out of order
    [99, 0, 0, 0, 0],                         # none at all
    [-7, -3, 0, 100, 100, -(1 << 31)],
    [0, 60, 100] + [0] * 400,                 # more of them than the gradient's last kernel looks through in one go
    [0] + [7 * i for i in range(1, 12)] + [-1] * 300,
    [1 << 30, 50, 20] + [61] * 300 + [90, 80],
    [3, 60, 60, 61] + [91] * 300,             # as many that do not fall
    list(range(5, 96)) + [95] * 257,
]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Hq,Hk,d", [(2, 2, 64), (6, 2, 128)])
@pytest.mark.parametrize("qs", STARTS)
def test_against_the_definition(qs, Hq, Hk, d, causal):
    n = 100
    g = torch.Generator("cuda").manual_seed(len(qs))
    rand = lambda h: torch.randn((h, n, d), generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v, do = rand(Hq), rand(Hk), rand(Hk), rand(Hq)
    st = torch.tensor(qs, dtype=torch.int32, device="cuda")
    clipped = [min(max(x, 0), n) for x in qs]
    scale = ela.default_scale(d)
    o, lse = torch.full_like(q, 7), torch.full((Hq, n), 7.0, device="cuda")
    ela.attn_fwd_packed(q, k, v, st, causal=causal, out=o, lse=lse)
    ref = packed(q, k, v, clipped, clipped, causal, scale)
    check(o, lse, ref)
    none = torch.isnan(ref[1][0])
    assert bool((o[:, none] == 7).all()) and bool((lse[:, none] == 7).all())
    for x in (q, k, v, do):
        x[:, none] = math.nan
    dq, dk, dv = (torch.full_like(x, 7) for x in (q, k, v))
    ela.attn_bwd_packed(q, k, v, o, lse, do, st, causal=causal, dq=dq, dk=dk, dv=dv)
    assert ela.last_device_error() == ela.ATTN_OK
    check_bwd((dq, dk, dv), *packed_bwd(q, k, v, o, lse, do, clipped, clipped, causal, scale))
    for x in (dq, dk, dv):
        assert bool((x[:, none] == 7).all())
