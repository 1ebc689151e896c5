"""What the packed and paged calls accept.  Without a device the checks of arguments pass on to the missing device, whose status
no refusal has; on a GPU real buffers get ATTN_OK and the right rows, and a workspace one byte short is refused."""
import pytest
import torch

import exact_long_sequence_gb300 as ela
from exact_long_sequence_gb300 import _build
from test_packed_arguments import bwd, fwd, i64, tree

NO_DEVICE = (ela.ATTN_ERR_NO_DEVICE, ela.ATTN_ERR_CUDA)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ela.load_library()


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up")
def test_accepted_without_a_device(lib):
    for call in (fwd, bwd):
        for good in (dict(), dict(Hq=64, Hk=1), dict(R=1, Nq=1, Nk=1), dict(d=128), dict(Hq=5, Hk=5), dict(scale=0.0), dict(scale=-3.0),
                     dict(Nq=1 << 29, Nk=1 << 28, Hq=2, Hk=2), dict(R=1 << 20)):
            assert call(lib, **good) in NO_DEVICE, good
    for good in (dict(Nk=1, ks=i64(64, -3)), dict(Hq=1, Hk=1, qs=i64(-5, 64)), dict(qs=i64(64, 256)), dict(ks=i64(64, 512), vs=i64(640, 64)),
                 dict(os_=i64(64, 1 << 20))):
        assert fwd(lib, **good) in NO_DEVICE, good
    for i in range(8):
        assert bwd(lib, st=[i64(72, 720) if j == i else None for j in range(8)]) in NO_DEVICE
    for good in (dict(), dict(mask=None), dict(page=1024, stride=0), dict(T=1), dict(T=1, R=1, most=1, pages=1), dict(Hq=128, Hk=2),
                 dict(page=16, most=1 << 26), dict(stride=1 << 40)):
        assert tree(lib, **good) in NO_DEVICE, good


def rand(seed, *shape):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(torch.bfloat16)


def room(size):
    assert size > 0
    return torch.empty(size, dtype=torch.uint8, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk,Nq,Nk", [(64, 1, 10, 10), (4, 2, 10, 1), (1, 1, 1, 1)])
def test_accepted_forms_of_packed_sequences(lib, Hq, Hk, Nq, Nk):
    d = 64
    q, k, v, do = rand(0, Hq, Nq, d), rand(1, Hk, Nk, d), rand(2, Hk, Nk, d), rand(3, Hq, Nq, d)
    qst, kst = (torch.tensor([0, 0, n], dtype=torch.int32, device="cuda") for n in (Nq, Nk))
    o, lse = torch.empty_like(q), torch.empty((Hq, Nq), device="cuda")
    want = ela.attn_fwd_packed(q, k, v, qst, kst)
    torch.cuda.synchronize()
    ws = room(lib.attn_fwd_packed_workspace_bytes(2, Nq, Nk, Hq, Hk, d))
    # axes of one are never stepped, whatever their strides are
    qs, ks = i64(Nq * d if Hq > 1 else -5, d if Nq > 1 else -3), i64(Nk * d if Hk > 1 else 0, d if Nk > 1 else 7)

    def forward(size):
        return lib.attn_fwd_packed(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), ks, qst.data_ptr(), kst.data_ptr(), o.data_ptr(),
                                   qs, lse.data_ptr(), 2, Nq, Nk, Hq, Hk, d, 0, 0.125, ws.data_ptr(), size, None)

    assert forward(ws.numel()) == ela.ATTN_OK
    assert forward(ws.numel() - 1) == ela.ATTN_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    want = ela.attn_bwd_packed(q, k, v, o, lse, do, qst, kst)
    torch.cuda.synchronize()
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = room(lib.attn_bwd_packed_workspace_bytes(2, Nq, Nk, Hq, Hk, d))

    def backward(size):
        return lib.attn_bwd_packed(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), ks, o.data_ptr(), qs, lse.data_ptr(),
                                   do.data_ptr(), qs, qst.data_ptr(), kst.data_ptr(), dq.data_ptr(), qs, dk.data_ptr(), ks, dv.data_ptr(),
                                   ks, 2, Nq, Nk, Hq, Hk, d, 0, 0.125, ws.data_ptr(), size, None)

    assert backward(ws.numel()) == ela.ATTN_OK
    assert backward(ws.numel() - 1) == ela.ATTN_ERR_INVALID_ARG
    torch.cuda.synchronize()
    # (at most one tile of keys to a sequence: dQ has one term and the same bits too)
    assert all(torch.equal(x, y) for x, y in zip((dq, dk, dv), want))
    assert ela.last_device_error() == ela.ATTN_OK


@pytest.mark.gpu
@pytest.mark.parametrize("page,stride", [(1024, 0), (16, 0), (32, 3)])
def test_accepted_forms_of_pages(lib, page, stride):
    """A table whose rows are one (stride 0), pages of the largest and the smallest size, and no mask."""
    R, Hq, Hk, T, d, pages, most = 2, 64, 1, 3, 64, 5, 3
    q, kc, vc = rand(0, R, Hq, T, d), rand(1, pages, Hk, page, d), rand(2, pages, Hk, page, d)
    rows = torch.tensor([[4, 0, 2], [4, 0, 2] if stride == 0 else [1, 3, 0]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([3 * page, page + 5], dtype=torch.int32, device="cuda")
    want = ela.attn_fwd_tree(q, kc, vc, rows, lens)
    o, lse = torch.empty_like(q), torch.empty((R, Hq, T), device="cuda")
    ws = room(lib.attn_fwd_tree_workspace_bytes(R, Hq, Hk, T, d))
    torch.cuda.synchronize()
    st = lib.attn_fwd_tree(q.data_ptr(), None, kc.data_ptr(), None, vc.data_ptr(), None, rows.data_ptr(), stride, lens.data_ptr(), None,
                           o.data_ptr(), None, lse.data_ptr(), R, Hq, Hk, T, pages, page, most, d, 0.125, ws.data_ptr(), ws.numel(), None)
    assert st == ela.ATTN_OK
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert ela.last_device_error() == ela.ATTN_OK
