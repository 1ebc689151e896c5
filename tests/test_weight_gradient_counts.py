"""Weight gradients of the query / key preparation as counts (GPU).

Inputs and upstream gradients are +-1, eps is 0 and no pair turns, so h = x and dw_j is the whole
number sum g_j x_j: one row left out, added twice or taken from a lane without a row shows as 1.
Bound: the norm is off by at most 2^-21 (rsqrt).  A sum passes through at most 64 additions: up to
12 rows of a lane (the work of these shapes dealt to some hundreds of warps), 3 over the row groups
of a warp, 12 warps, 5 rows of 152 CTAs and 32 in the finishing kernel.  So dw is off by at
most n (2^-21 + 64 * 2^-24) = 72 n 2^-24, below 1/2 for n <= 100000 even if every error had one
sign; and the sums are of whole numbers where rsqrt(1) is 1.
"""
import pytest
import torch

import exact_long_sequence_gb300 as ela
from exact_long_sequence_gb300 import _build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    _build.build()
    ela.load_library()


@pytest.mark.parametrize("d,Hq,Hk,B,N", [
    (64, 1, 4, 2, 4099),    # several tokens a step, the last step short
    (64, 1, 1, 3, 8191),
    (64, 9, 3, 3, 333),
    (64, 17, 1, 1, 1200),
    (128, 2, 1, 3, 3333),
    (128, 8, 2, 1, 2500),   # whole tokens per warp
    (128, 5, 5, 2, 2001),
    (128, 3, 1, 1, 1),
])
def test_every_row_counts_once(d, Hq, Hk, B, N):
    assert B * N * max(Hq, Hk) <= 100000
    g = torch.Generator("cuda").manual_seed(d + N)

    def signs(*shape):
        return (torch.randint(0, 2, shape, generator=g, device="cuda") * 2 - 1).to(torch.bfloat16)

    q, k, gq, gk = signs(B, Hq, N, d), signs(B, Hk, N, d), signs(B, Hq, N, d), signs(B, Hk, N, d)
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(N, dtype=torch.int32, device="cuda")
    inv = torch.ones(d // 2, dtype=torch.float64, device="cuda")
    _, _, dwq, dwk = ela.qk_norm_rope_bwd(gq, gk, q, k, pos, inv, w, w, eps=0.0)
    for got, x, dy in ((dwq, q, gq), (dwk, k, gk)):
        want = (x.double() * dy.double()).sum((0, 1, 2))
        assert ((got.double() - want).abs() < 0.5).all()
