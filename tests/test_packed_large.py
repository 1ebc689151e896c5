"""Packed and paged calls on tensors of more than 2^31 elements or on 2^24 keys, and the gradient in its most turns (GPU).
Only some sequences, at the ends and in the middle, are compared with the definition."""
import math

import pytest
import torch

import exact_long_sequence_gb300 as ela
from packed_ref import bits, check, check_bwd, packed, packed_bwd, starts, tree
from test_tree import random_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def rand(seed, *shape):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda", dtype=torch.bfloat16)


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("token_major", [True, False])
def test_sequences(token_major):
    Hq, Hk, d = 32, 4, 128
    lens = torch.randint(1, 3001, (410,), generator=torch.Generator().manual_seed(1)).tolist()
    lens[0], lens[200], lens[-1] = 2047, 1, 2500
    qs = starts(lens)
    N = qs[-1]
    assert Hq * N * d > 1 << 31 and 8 * N * Hq * d > 32 * 150e6

    def tensor(seed, h):
        return rand(seed, N, h, d).transpose(0, 1) if token_major else rand(seed, h, N, d)

    q, k, v, do = tensor(0, Hq), tensor(1, Hk), tensor(2, Hk), tensor(3, Hq)
    st = dev(qs)
    scale = ela.default_scale(d)
    o, lse = ela.attn_fwd_packed(q, k, v, st, causal=True, out=torch.empty_like(q))
    grads = ela.attn_bwd_packed(q, k, v, o, lse, do, st, causal=True, dq=torch.empty_like(q))
    assert ela.last_device_error() == ela.ATTN_OK
    for s in (0, 1, 199, 200, 201, 408, 409):
        own = slice(qs[s], qs[s + 1])
        a = [x[:, own] for x in (q, k, v, o, lse, do)]
        one = [0, lens[s]]
        check(a[3], a[4], packed(a[0], a[1], a[2], one, one, True, scale))
        check_bwd([x[:, own] for x in grads], *packed_bwd(*a, one, one, True, scale))


@pytest.mark.parametrize("token_major", [True, False])
def test_pages(token_major):
    Hq, Hk, d, T, page, pages = 16, 8, 128, 40, 64, 36000
    kc, vc = ((rand(s, pages, page, Hk, d).transpose(1, 2) if token_major else rand(s, pages, Hk, page, d)) for s in (1, 2))
    assert kc.numel() > 1 << 31
    lens = [12011, 40, 20000, 641]
    R = len(lens)
    table = torch.randint(0, pages, (R, 313), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    table[0, :3] = torch.tensor([pages - 1, 0, pages - 2])
    table[3, 10] = pages - 1
    table = table.cuda()
    q = rand(3, R, Hq, T, d)
    seen = random_tree(torch.Generator().manual_seed(4), R, T)
    out, lse = ela.attn_fwd_tree(q, kc, vc, table, dev(lens), bits(seen).cuda())
    assert ela.last_device_error() == ela.ATTN_OK
    check(out, lse, tree(q, kc, vc, table, lens, seen, ela.default_scale(d)))


@pytest.mark.parametrize("d", [64, 128])
def test_many_keys(d):
    """A request whose table names four pages again and again: the softmax over them once, and the log-sum-exp moved by the
    logarithm of how often.  A piece's rows are sums of 2^17 keys' terms in fp32, in steps of 16: off by at most 2^13 roundings of
    2^-24, which check()'s 2^-11 of the terms' sum holds."""
    page, times = 1024, 4096
    kc, vc, q = rand(1, 4, 1, page, d), rand(2, 4, 1, page, d), rand(3, 1, 4, 1, d)
    table = torch.arange(4, dtype=torch.int32, device="cuda").repeat(times)[None].contiguous()
    out, lse = ela.attn_fwd_tree(q, kc, vc, table, dev([4 * page * times]))
    assert ela.last_device_error() == ela.ATTN_OK
    seen = torch.ones((1, 1, 1), dtype=torch.bool, device="cuda")
    ro, rl, ra = tree(q, kc, vc, table[:, :4], [4 * page], seen, ela.default_scale(d))
    check(out, lse, (ro, rl + math.log(times), ra))
