"""Stream order of the packed and paged calls (GPU): everything that the caller's stream holds is done before a call starts.

A programmatic dependent waits, at its `griddepcontrol.wait`, for the grid before it.  Where that grid is itself a
programmatic dependent which needs nothing of the grids before it and does not wait for them, they may still run.  So
the first launch of a call has to be a plain one.  Shown on the graph of a captured call, which runs nothing, and by calls
behind such a grid.
"""
import ctypes
import subprocess

import pytest
import torch

import exact_long_sequence_gb300 as ela
from exact_long_sequence_gb300 import _build

pytestmark = pytest.mark.gpu
D, HQ, HK = 64, 4, 2

KERNELS = r"""
#include <cuda_runtime.h>
// Lets the next grid start at once, waits some milliseconds (a bounded number of naps), then fills x.
__global__ void late_fill(unsigned short* x, size_t n, unsigned short v, int naps) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = 0; i < naps; ++i) __nanosleep(1000);
    for (size_t i = threadIdx.x; i < n; i += blockDim.x) x[i] = v;
}
// A grid that needs nothing of those before it, and waits for none.
__global__ void beside(int* y) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) *y += 1;
}
extern "C" int before_the_call(void* x, size_t n, int v, int naps, void* y, cudaStream_t stream) {
    late_fill<<<1, 1024, 0, stream>>>(static_cast<unsigned short*>(x), n, static_cast<unsigned short>(v), naps);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, beside, static_cast<int*>(y));
}
"""


def rand(seed, *shape):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(torch.bfloat16)


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def packed(n):
    """A call on given buffers, and the tensor of its that the work before it fills; up to 640 keys it is one launch."""
    q, k, v, st = rand(1, HQ, n, D), rand(2, HK, n, D), rand(3, HK, n, D), dev([0, n // 3, n])
    out, lse = torch.empty_like(q), torch.empty((HQ, n), device="cuda")
    ws = torch.empty(ela.packed_workspace_bytes(2, n, n, HQ, HK, D), dtype=torch.uint8, device="cuda")
    return lambda: ela.attn_fwd_packed(q, k, v, st, causal=True, out=out, lse=lse, workspace=ws), v


def gradient(n):
    q, k, v, do, st = rand(1, HQ, n, D), rand(2, HK, n, D), rand(3, HK, n, D), rand(4, HQ, n, D), dev([0, n // 3, n])
    o, lse = ela.attn_fwd_packed(q, k, v, st, causal=True)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = torch.empty(ela.packed_bwd_workspace_bytes(2, n, n, HQ, HK, D), dtype=torch.uint8, device="cuda")
    return lambda: ela.attn_bwd_packed(q, k, v, o, lse, do, st, causal=True, dq=dq, dk=dk, dv=dv, workspace=ws), o


def drafts(pages):
    R, T, page = 2, 3, 16
    q, kc, vc = rand(1, R, HQ, T, D), rand(2, pages, HK, page, D), rand(3, pages, HK, page, D)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(R, pages).contiguous()
    lens = dev([pages * page, 40])
    out, lse = torch.empty_like(q), torch.empty((R, HQ, T), device="cuda")
    ws = torch.empty(ela.tree_workspace_bytes(R, HQ, HK, T, D), dtype=torch.uint8, device="cuda")
    return lambda: ela.attn_fwd_tree(q, kc, vc, table, lens, out=out, lse=lse, workspace=ws), vc


CALLS = {"packed, one launch": (packed, 300), "packed, two launches": (packed, 3000), "gradient": (gradient, 700),
         "drafts, one launch": (drafts, 10), "drafts, two launches": (drafts, 200)}


def captured_edges(work):
    """(from, to, programmatic) of the graph of `work` on a stream of its own."""
    cu = ctypes.CDLL("libcuda.so.1")
    vp = ctypes.c_void_p
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    stream.synchronize()
    graph, count = vp(), ctypes.c_size_t()
    with torch.cuda.stream(stream):
        assert cu.cuStreamBeginCapture_v2(vp(stream.cuda_stream), 2) == 0  # relaxed
        try:
            work()
        finally:
            assert cu.cuStreamEndCapture(vp(stream.cuda_stream), ctypes.byref(graph)) == 0
    try:
        assert cu.cuGraphGetEdges_v2(graph, None, None, None, ctypes.byref(count)) == 0
        src, to, data = (vp * count.value)(), (vp * count.value)(), (ctypes.c_uint8 * 8 * count.value)()
        assert cu.cuGraphGetEdges_v2(graph, src, to, data, ctypes.byref(count)) == 0
        return [(a, b, data[i][2] != 0) for i, (a, b) in enumerate(zip(src, to))]
    finally:
        cu.cuGraphDestroy(graph)


@pytest.mark.parametrize("name", CALLS)
def test_the_first_launch_waits_for_all_before(name):
    make, size = CALLS[name]
    call, filled = make(size)
    call()
    torch.cuda.synchronize()

    def work():
        filled.mul_(1)
        call()

    edges = captured_edges(work)
    inner = {b for _, b, _ in edges}
    first = [e for e in edges if e[0] not in inner]  # from the product before the call
    assert len(first) == 1 and not first[0][2]
    assert len(edges) == {"one launch": 1, "two launches": 2, "gradient": 3}[name.split(", ")[-1]]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    at = tmp_path_factory.mktemp("order")
    (at / "before.cu").write_text(KERNELS)
    so = at / "before.so"
    subprocess.run([_build.nvcc(), "-shared", "-O2", "-Xcompiler", "-fPIC", str(at / "before.cu"), "-o", str(so)] + _build.ARCH,
                   check=True)
    lib = ctypes.CDLL(str(so))
    lib.before_the_call.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]
    return lib


@pytest.mark.parametrize("name", CALLS)
def test_behind_a_grid_that_does_not_wait(lib, name):
    """The call reads what the first of two grids writes late, while the second, which did not wait for it, is long done."""
    make, size = CALLS[name]
    call, filled = make(size)
    filled.fill_(2)
    want = [x.clone() for x in call()]
    y = torch.zeros(1, dtype=torch.int32, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for naps in (0, 2000):
        filled.fill_(5)
        torch.cuda.synchronize()
        assert lib.before_the_call(filled.data_ptr(), filled.numel(), 0x4000, naps, y.data_ptr(), stream) == 0  # 2 in bf16
        got = call()
        torch.cuda.synchronize()
        assert bool((filled == 2).all())
        for g, w in list(zip(got, want))[1 if name == "gradient" else 0:]:  # (dQ: an order of sums)
            assert torch.equal(g, w)
    assert ela.last_device_error() == ela.ATTN_OK
