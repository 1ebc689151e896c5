"""Shared-prefix attention where single keys decide the result (GPU).

With random inputs over long ranges O is an average close to zero, and a wrong or missing tile hardly
moves it.  Here every row has a key of its own, c times its query, that has all but e^-10 of the weight:
its score is c |q|^2 / sqrt(d), 56 for d = 128 and 40 for d = 64 with c = 5, while all others together reach about
log(keys) + 1/2 < 16 and a foreign row's key c times a normal number.  So O is that key's V, and a
key read from elsewhere, skipped or counted twice is off by the size of V or, in the log-sum-exp,
by the score.  The bounds are those of test_prefix, which take the larger scores into account.
"""
import pytest
import torch

import exact_long_sequence_gb300 as ela
from exact_long_sequence_gb300 import _build

from test_prefix import check

pytestmark = pytest.mark.gpu
C_NEEDLE = 5.0


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    _build.build()
    ela.load_library()


def draw(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def needle(q):
    return (C_NEEDLE * q.float()).to(torch.bfloat16)


def found(out, v):
    """O is the needle's V: the two differ by the P and O roundings and the other keys' weight of e^-10."""
    assert ((out.float() - v.float()).abs() <= 2.0 ** -6 * (1 + v.float().abs())).all()


@pytest.mark.parametrize("R,Hk,G,d,P", [
    (64, 8, 4, 128, 16384),   # two rows for each tile of a head; two query tiles
    (64, 4, 4, 64, 40000),    # 313 tiles, 256 needles
    (30, 8, 4, 128, 15360),   # 120 rows: one query tile, the chains take turns
    (15, 3, 8, 64, 15301),    # ... and a tail
    (200, 1, 8, 128, 20001),  # seven row blocks of one key head
])
def test_every_tile_of_the_prefix(R, Hk, G, d, P):
    g = torch.Generator("cuda").manual_seed(P)
    q, kp, vp = draw(g, R, Hk * G, 1, d), draw(g, Hk, P, d), draw(g, Hk, P, d)
    rows = R * G
    # spread over all tiles, each at its own place in the tile
    at = (torch.arange(rows, device="cuda") * P // rows + torch.arange(rows, device="cuda") * 37 % max(1, P // rows)).clamp(max=P - 1)
    assert at.unique().numel() == min(rows, P) and (P + 127) // 128 <= rows * 2
    for h in range(Hk):
        mine = q[:, h * G:(h + 1) * G, 0].reshape(rows, d)
        kp[h, at] = needle(mine)
    s = dict(q=q, k_prefix=kp, v_prefix=vp)
    out, lse = ela.attn_fwd_prefix(**s)
    check(s, out, lse)
    for h in range(Hk):
        found(out[:, h * G:(h + 1) * G, 0].reshape(rows, d), vp[h, at])


@pytest.mark.parametrize("R,Hk,G,d,P,C", [
    (200, 1, 4, 128, 0, 512),    # the own-keys kernel alone
    (200, 1, 4, 64, 700, 512),   # ... and beside a prefix
    (64, 2, 4, 128, 700, 2048),  # items of the prefix kernel
    (5, 1, 3, 64, 300, 1030),
])
def test_every_step_of_the_own_keys(R, Hk, G, d, P, C):
    g = torch.Generator("cuda").manual_seed(C)
    q, ko, vo = draw(g, R, Hk * G, 1, d), draw(g, R, Hk, C, d), draw(g, R, Hk, C, d)
    lens = [C - (r * 7) % 16 for r in range(R)]
    at = torch.tensor([[((r * G + x) * 61) % lens[r] for x in range(G)] for r in range(R)], device="cuda")
    for r in range(R):
        assert at[r].unique().numel() == G
        for h in range(Hk):
            ko[r, h, at[r]] = needle(q[r, h * G:(h + 1) * G, 0])
    s = dict(q=q, k_own=ko, v_own=vo, own_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if P:
        s["k_prefix"], s["v_prefix"] = draw(g, Hk, P, d), draw(g, Hk, P, d)
    out, lse = ela.attn_fwd_prefix(**s)
    check(s, out, lse)
    for r in range(R):
        for h in range(Hk):
            found(out[r, h * G:(h + 1) * G, 0], vo[r, h, at[r]])


def test_offsets_past_32_bits_decide():
    """The keys that decide lie past 2^31 elements, in the prefix and in the own caches, read by either kernel."""
    Hk, d, P = 8, 128, 2_100_000
    far = [P - 1, P - 2, P - 20000]
    assert all((7 * P + x) * d >= 2 ** 31 for x in far)
    g = torch.Generator("cuda").manual_seed(21)
    kp, vp = (torch.empty(Hk, P, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for x in (kp, vp):
        for h in range(Hk):
            x[h] = draw(g, P, d)
    q = draw(g, 3, Hk, 1, d)
    for r, x in enumerate(far):
        kp[7, x] = needle(q[r, 7, 0])
    out, lse = ela.attn_fwd_prefix(q, kp, vp)
    check(dict(q=q[:, 7:], k_prefix=kp[7:], v_prefix=vp[7:]), out[:, 7:], lse[:, 7:])
    found(out[:, 7, 0], vp[7, far])
    # the same memory as own caches of two requests with four heads each: the far keys are request 1's, head 3's
    ko, vo = kp.view(2, 4, P, d), vp.view(2, 4, P, d)
    near = draw(g, 4, 64, d)
    for r, x in enumerate(far):
        q2 = draw(g, 2, 4, 1, d)
        q2[1, 3] = q[r, 7]
        for lens in ([100, P], [P, P]):
            n = torch.tensor(lens, dtype=torch.int32, device="cuda")
            for pre in ({}, dict(k_prefix=near, v_prefix=near)):  # the own-keys kernel, items of the prefix kernel
                out, lse = ela.attn_fwd_prefix(q2, k_own=ko, v_own=vo, own_lens=n, **pre)
                assert ela.last_device_error() == ela.ATTN_OK
                found(out[1, 3, 0], vo[1, 3, x])
                score = (q2[1, 3, 0].double() * ko[1, 3, x].double()).sum() / d ** 0.5
                assert abs(lse[1, 3, 0].double() - score) <= 2.0 ** -10
