"""The packed and paged calls on given streams, inside a captured graph, and run after run on one workspace (GPU).

dQ is summed in the order in which key tiles are done: equal calls may differ by the fp32 sums' rounding (64 tiles: 2^-18 of
the largest term) and then by one bf16 step (2^-7 of the value).  Everything else is the same bit for bit.
"""
import pytest
import torch

import exact_long_sequence_gb300 as ela

pytestmark = pytest.mark.gpu


def draw(seed, *shape):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def lengths(seed, n, hi):
    lens = torch.randint(1, hi, (n,), generator=torch.Generator().manual_seed(seed))
    return torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)]).to(torch.int32).cuda(), int(lens.sum())


def forward(seed, hi=4000, n=5):
    st, N = lengths(seed, n, hi)
    q, k, v = draw(seed, 8, N, 128), draw(seed + 1, 2, N, 128), draw(seed + 2, 2, N, 128)
    return lambda stream=None, workspace=None: ela.attn_fwd_packed(q, k, v, st, causal=True, stream=stream, workspace=workspace)


def short(seed):
    return forward(seed, hi=60, n=9)


def backward(seed):
    st, N = lengths(seed, 5, 2000)
    q, k, v, do = draw(seed, 6, N, 128), draw(seed + 1, 2, N, 128), draw(seed + 2, 2, N, 128), draw(seed + 3, 6, N, 128)
    o, lse = ela.attn_fwd_packed(q, k, v, st, causal=True)
    torch.cuda.synchronize()
    return lambda stream=None, workspace=None: ela.attn_bwd_packed(q, k, v, o, lse, do, st, causal=True, stream=stream, workspace=workspace)


def drafts(seed, T=8):
    R, pages, page = 24, 900, 64
    q, kc, vc = draw(seed, R, 8, T, 128), draw(seed + 1, pages, 2, page, 128), draw(seed + 2, pages, 2, page, 128)
    g = torch.Generator().manual_seed(seed)
    table = torch.randint(0, pages, (R, 40), generator=g).to(torch.int32).cuda()
    lens = torch.randint(T, 40 * page, (R,), generator=g).to(torch.int32).cuda()
    return lambda stream=None, workspace=None: ela.attn_fwd_tree(q, kc, vc, table, lens, stream=stream, workspace=workspace)


def one(seed):
    return drafts(seed, 1)


CALLS = {"forward": forward, "short": short, "backward": backward, "drafts": drafts, "one": one}


def same(got, want):
    first = 0
    if len(got) == 3:  # dQ
        a, b = got[0].float(), want[0].float()
        assert bool(((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -18 * b.abs().max()).all())
        first = 1
    assert all(torch.equal(x, y) for x, y in zip(got[first:], want[first:]))


@pytest.mark.parametrize("name", CALLS)
def test_side_by_side_without_a_wait(name):
    a, b = CALLS[name](1), CALLS[name](100)
    want = a(), b()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        got = [a() for _ in range(3)][-1], b(side), a()
        torch.cuda.synchronize()
        for x, w in zip(got, (want[0], want[1], want[0])):
            same(x, w)
    assert ela.last_device_error() == ela.ATTN_OK


def test_on_a_stream_that_joined_a_capture():
    calls = [make(1) for make in CALLS.values()]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = [(call(), call(side), call(side)) for call in calls]
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for each, w in zip(got, want):
            for x in each:
                same(x, w)
    assert ela.last_device_error() == ela.ATTN_OK


def test_one_workspace_call_after_call():
    """Every kind of call after every other on one workspace, which each leaves full of its own: launches that set up beside
    the one before must not touch it early."""
    calls = [make(7) for make in CALLS.values()]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    work = torch.full((1 << 30,), 255, dtype=torch.uint8, device="cuda")  # (NaN in fp32, -1 in integers)
    order = [(i, j) for i in range(len(calls)) for j in range(len(calls))]
    got = [(x, calls[x](workspace=work)) for pair in order for x in pair]
    torch.cuda.synchronize()
    for x, result in got:
        same(result, want[x])
    assert ela.last_device_error() == ela.ATTN_OK
