"""The kernel for own keys of few rows, at shapes that reach it, and the same calls as items of the
prefix kernel (GPU).  The own-keys kernel works where there is no prefix or there are more sequences
(requests times key heads) than SMs; the other cases here keep below that."""
import pytest
import torch

import exact_long_sequence_gb300 as ela
from exact_long_sequence_gb300 import _build

from test_prefix import check, make

pytestmark = pytest.mark.gpu
# R, Hq, Hk, P: the own-keys kernel alone, beside a prefix, and items of the prefix kernel
PATHS = [(6, 8, 2, 0), (170, 4, 1, 300), (6, 8, 2, 300)]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    _build.build()
    ela.load_library()
    assert torch.cuda.get_device_properties(0).multi_processor_count < 170


def lengths(R, C):
    return [(37 * r + 11) % (C + 1) for r in range(R)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0, 1e-30])
@pytest.mark.parametrize("path", PATHS, ids=str)
def test_any_finite_scale(path, scale, d):
    R, Hq, Hk, P = path
    s = make(R, Hq, Hk, 1, d, P, 150, lengths(R, 150), seed=3)
    out, lse = ela.attn_fwd_prefix(**s, scale=scale)
    check(s, out, lse, scale=scale, requests=range(0, R, 7) if R > 20 else None)


@pytest.mark.parametrize("path", [(64, 8, 2, 0), (170, 4, 1, 300), (8, 8, 2, 300)], ids=str)
def test_scores_that_rise_move_the_reference_maximum(path):
    """Scores of a row rise by 0, 14, 28 or 57 (or fall) from one step of 16 keys to the next; the reference moves
    where they pass it by 32 log 2 = 22, also more than once within one worker's stretch: in the first shape a
    stretch is 18 steps or more (64 x 2 sequences of 170 steps on 1216 warps), in the second 23, in the third tiles of 128 keys."""
    R, Hq, Hk, P = path
    d, C = 128, 2720
    s = make(R, Hq, Hk, 1, d, P, C, [C - r % 40 for r in range(R)], seed=5)
    G = Hq // Hk
    for h in range(Hk):
        base = torch.randn(R, d, generator=torch.Generator("cuda").manual_seed(h), device="cuda")
        base = base / base.norm(dim=-1, keepdim=True) * d ** 0.5
        for x, f in enumerate((1.0, -1.0, 0.5, 2.0)[:G]):
            s["q"][:, h * G + x, 0] = (f * base).to(torch.bfloat16)
        step = torch.arange(C, device="cuda") // 16 % 20  # 28.3 a step for f = 1, for 20 steps, then again
        keys = 2.5 * step[None, :, None] * base[:, None] + torch.randn(R, C, d, generator=torch.Generator("cuda").manual_seed(9 + h),
                                                                       device="cuda")
        s["k_own"][:, h] = keys.to(torch.bfloat16)
    for r in range(R):
        s["k_own"][r, :, s["own_lens"][r]:] = float("nan")
    out, lse = ela.attn_fwd_prefix(**s)
    check(s, out, lse, requests=range(0, R, 13) if R > 20 else None)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("R,Hq,Hk,T,d,P", [
    (6, 8, 2, 3, 128, 0), (170, 4, 1, 3, 64, 300), (6, 8, 2, 3, 128, 300),
    (5, 20, 2, 3, 64, 0),    # 30 rows in blocks of 15
    (3, 16, 2, 17, 64, 100),  # 136 rows a request
])
def test_a_key_that_a_token_does_not_see_does_not_reach_it(R, Hq, Hk, T, d, P, value):
    """The last new token's K is not finite: the tokens before it give the same bits as without it."""
    C = 200
    lens = [T + (23 * r) % (C - T + 1) for r in range(R)]
    s = make(R, Hq, Hk, T, d, P, C, lens, seed=8)
    clean = [x.clone() for x in ela.attn_fwd_prefix(**s)]
    for r in range(R):
        s["k_own"][r, :, lens[r] - 1] = value
    out, lse = ela.attn_fwd_prefix(**s)
    assert torch.equal(out[:, :, :-1], clean[0][:, :, :-1]) and torch.equal(lse[:, :, :-1], clean[1][:, :, :-1])
    assert torch.isfinite(clean[0]).all() and torch.isfinite(clean[1]).all()
    if value != value:
        assert out[:, :, -1].isnan().all() and lse[:, :, -1].isnan().all()
