"""What the packed and paged calls refuse, on the CPU: nothing is launched, and nothing is read through the addresses."""
import ctypes

import pytest
import torch

import exact_long_sequence_gb300 as ela
from exact_long_sequence_gb300 import _build

OK, INVALID, UNSUPPORTED, MISALIGNED = ela.ATTN_OK, ela.ATTN_ERR_INVALID_ARG, ela.ATTN_ERR_UNSUPPORTED, ela.ATTN_ERR_MISALIGNED
A = 0x10000  # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ela.load_library()


def i64(*x):
    return (ctypes.c_int64 * len(x))(*x)


def fwd(lib, q=A, k=A, v=A, qst=A, kst=A, o=A, lse=A, R=2, Nq=10, Nk=10, Hq=4, Hk=2, d=64, scale=0.1, ws=A, qs=None, ks=None, vs=None, os_=None):
    # (a workspace of no bytes: with a device too, the call ends before a launch)
    return lib.attn_fwd_packed(q, qs, k, ks, v, vs, qst, kst, o, os_, lse, R, Nq, Nk, Hq, Hk, d, 1, scale, ws, 0, None)


def bwd(lib, t=(A,) * 8, lse=A, qst=A, kst=A, R=2, Nq=10, Nk=10, Hq=4, Hk=2, d=64, scale=0.1, ws=A, st=(None,) * 8):
    q, k, v, o, do, dq, dk, dv = t
    return lib.attn_bwd_packed(q, st[0], k, st[1], v, st[2], o, st[3], lse, do, st[4], qst, kst, dq, st[5], dk, st[6], dv, st[7],
                               R, Nq, Nk, Hq, Hk, d, 1, scale, ws, 0, None)


def tree(lib, q=A, k=A, v=A, table=A, stride=4, lens=A, mask=A, o=A, lse=A, R=2, Hq=4, Hk=2, T=3, pages=5, page=16, most=4, d=64, scale=0.1,
         ws=A, qs=None, ks=None):
    return lib.attn_fwd_tree(q, qs, k, ks, v, None, table, stride, lens, mask, o, None, lse, R, Hq, Hk, T, pages, page, most, d, scale, ws,
                             0, None)


def passes(status):
    """The checks passed: what is missing then is a device, or room in the workspace."""
    return status in (ela.ATTN_ERR_NO_DEVICE, ela.ATTN_ERR_CUDA, INVALID)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_shapes(lib, call):
    for bad in (dict(R=0), dict(Nq=0), dict(Nk=0), dict(Hq=0), dict(Hk=0), dict(Hk=3), dict(Hq=-4), dict(Nq=(1 << 31) - 1),
                dict(Nk=1 << 30), dict(Hq=1 << 20, Hk=1 << 15, Nq=1 << 12), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(lib, **bad) == INVALID, bad
    for bad in (dict(d=96), dict(d=0), dict(Hq=65, Hk=1), dict(Hq=260, Hk=2)):
        assert call(lib, **bad) == UNSUPPORTED, bad
    assert passes(call(lib, Hq=64, Hk=1))


def test_null_and_misaligned(lib):
    for x in ("q", "k", "v", "qst", "kst", "o", "lse", "ws"):
        assert fwd(lib, **{x: None}) == INVALID, x
    for x in ("q", "k", "v", "o", "ws"):
        assert fwd(lib, **{x: A + 8}) == MISALIGNED, x
    for x in ("qst", "kst", "lse"):
        assert fwd(lib, **{x: A + 2}) == MISALIGNED, x
    for i in range(8):
        assert bwd(lib, t=[None if j == i else A for j in range(8)]) == INVALID
        assert bwd(lib, t=[A + 8 if j == i else A for j in range(8)]) == MISALIGNED
    for x in ("lse", "qst", "kst", "ws"):
        assert bwd(lib, **{x: None}) == INVALID
        assert bwd(lib, **{x: A + 2}) == MISALIGNED
    for x in ("q", "k", "v", "table", "lens", "o", "lse", "ws"):
        assert tree(lib, **{x: None}) == INVALID, x
    for x in ("q", "k", "v", "o", "ws"):
        assert tree(lib, **{x: A + 8}) == MISALIGNED, x
    for x in ("table", "lens", "mask", "lse"):
        assert tree(lib, **{x: A + 1}) == MISALIGNED, x


def test_strides(lib):
    for x in ("qs", "ks", "vs", "os_"):
        assert fwd(lib, **{x: i64(64, 260)}) == MISALIGNED
        assert fwd(lib, **{x: i64(64, 0)}) == INVALID
        assert fwd(lib, **{x: i64(-64, 256)}) == INVALID
        assert fwd(lib, **{x: i64(1 << 40, 256)}) == INVALID
    assert passes(fwd(lib, Nk=1, ks=i64(64, -3)))  # an axis of one is never stepped
    for i in range(8):
        assert bwd(lib, st=[i64(64, 260) if j == i else None for j in range(8)]) == MISALIGNED
        assert bwd(lib, st=[i64(0, 256) if j == i else None for j in range(8)]) == INVALID
    assert tree(lib, qs=i64(1024, 64, 0)) == INVALID
    assert tree(lib, ks=i64(2048, 64, 12)) == MISALIGNED


def test_tree_shapes(lib):
    for bad in (dict(R=0), dict(T=0), dict(pages=0), dict(most=0), dict(page=0), dict(Hk=3), dict(stride=-1), dict(scale=float("nan")),
                dict(T=1 << 29), dict(most=1 << 28), dict(pages=(1 << 31) - 1)):
        assert tree(lib, **bad) == INVALID, bad
    for bad in (dict(d=32), dict(Hq=130, Hk=2), dict(page=8), dict(page=48), dict(page=2048)):
        assert tree(lib, **bad) == UNSUPPORTED, bad
    assert passes(tree(lib, mask=None)) and passes(tree(lib, page=1024, stride=0))


def test_workspace_of_an_invalid_shape_is_none(lib):
    assert lib.attn_fwd_packed_workspace_bytes(0, 1, 1, 1, 1, 64) == 0
    assert lib.attn_fwd_packed_workspace_bytes(1, 1, 1, 3, 2, 64) == 0
    assert lib.attn_bwd_packed_workspace_bytes(1, 1, 1, 1, 1, 65) == 0
    assert lib.attn_fwd_tree_workspace_bytes(1, 128, 1, 1, 64) == 0


def test_binding_refuses_on_the_cpu(lib):
    q, st = torch.zeros(2, 5, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        ela.attn_fwd_packed(q, q, q, st)
    with pytest.raises(ValueError):
        ela.attn_bwd_packed(q, q, q, q, torch.zeros(2, 5), q, st)
    with pytest.raises(ValueError):
        ela.attn_fwd_tree(q[None], q[None], q[None], st[None], st)


@pytest.mark.gpu
def test_binding_refusals():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    q, k, st, lse = z(4, 10, 64), z(2, 10, 64), torch.tensor([0, 10], dtype=torch.int32, device="cuda"), z(4, 10, dt=torch.float32)
    bad_fwd = [dict(q=q.float()), dict(q=q[..., :32]), dict(q=z(3, 10, 64)), dict(k=z(2, 10, 128)), dict(v=z(2, 9, 64)), dict(v=k.cpu()),
               dict(q_starts=st.long()), dict(q_starts=st[:1]), dict(q_starts=st.cpu()), dict(q_starts=st[None]), dict(k_starts=z(3, dt=torch.int32)),
               dict(out=z(4, 9, 64)), dict(out=z(4, 10, 128)[..., ::2]), dict(lse=z(4, 11, dt=torch.float32)), dict(lse=lse.double()),
               dict(workspace=z(4, dt=torch.float32)), dict(workspace=z(16, dt=torch.uint8)), dict(q=z(4, 10, 72)[..., :64]), dict(scale=float("nan"))]
    for change in bad_fwd:
        a = dict(q=q, k=k, v=k, q_starts=st)
        a.update(change)
        if "q" in change and change["q"].shape == (4, 10, 64) and change["q"].dtype == torch.bfloat16:
            ela.attn_fwd_packed(**a)  # (rows 72 apart are fine)
            continue
        with pytest.raises((ValueError, ela.AttnError)):
            ela.attn_fwd_packed(**a)
    for change in (dict(lse=None), dict(lse=lse.half()), dict(do=k), dict(o=q.float()), dict(dq=k), dict(dk=q), dict(dv=z(2, 10, 32)),
                   dict(workspace=z(16, dt=torch.uint8))):
        a = dict(q=q, k=k, v=k, o=q, lse=lse, do=q, q_starts=st)
        a.update(change)
        with pytest.raises((ValueError, ela.AttnError)):
            ela.attn_bwd_packed(**a)
    qt, kc = z(2, 4, 3, 64), z(5, 2, 16, 64)
    table, lens, mask = z(2, 4, dt=torch.int32), z(2, dt=torch.int32), z(2, 3, 1, dt=torch.int32)
    ela.attn_fwd_tree(qt, kc, kc, table, lens, mask)
    for change in (dict(q=qt[0]), dict(k_pages=kc[0]), dict(v_pages=z(4, 2, 16, 64)), dict(page_table=table.long()), dict(page_table=table[:1]),
                   dict(page_table=table.t().contiguous().t()), dict(lens=lens[:1]), dict(lens=lens.float()), dict(tree_mask=mask[..., 0]),
                   dict(tree_mask=mask.long()), dict(tree_mask=z(2, 3, 2, dt=torch.int32)), dict(k_pages=z(5, 2, 24, 64), v_pages=z(5, 2, 24, 64)),
                   dict(out=z(2, 4, 2, 64)), dict(lse=z(2, 4, dt=torch.float32)), dict(workspace=z(8, dt=torch.uint8))):
        a = dict(q=qt, k_pages=kc, v_pages=kc, page_table=table, lens=lens, tree_mask=mask)
        a.update(change)
        with pytest.raises((ValueError, ela.AttnError)):
            ela.attn_fwd_tree(**a)
    assert ela.last_device_error() == ela.ATTN_OK
