"""Where the binding takes memory for a call on a given stream.

The caching allocator hands a freed block out again in the order of the stream it belongs to.  A
buffer for a call on another stream must come from that stream's memory: a block of the current
stream may still be in use by that stream's earlier work.  What the caller gets back is marked as
used by the caller's stream.  On the CPU the allocator, the streams and the library are stand-ins
that record what is asked of them; on the GPU calls on two streams run side by side without a wait.
"""
import contextlib
import types

import pytest
import torch

import exact_long_sequence_gb300 as ela
from exact_long_sequence_gb300 import _build

gpu = pytest.mark.gpu
DEVICE = torch.device("cuda", 0)


class Tensor:
    """What the binding asks of a contiguous CUDA tensor."""

    is_cuda = True
    device = DEVICE

    def __init__(self, shape, dtype, made_on=None):
        self.shape, self.dtype, self.made_on, self.used_on = torch.Size(shape), dtype, made_on, []

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 0x1000

    def is_pinned(self):
        return False

    def unsqueeze(self, dim):
        return Tensor((1, *self.shape), self.dtype)

    def record_stream(self, stream):
        self.used_on.append(stream)


class Library:
    """Every query answers 4096 bytes, every call succeeds; the streams of the calls are kept."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_bytes"):
                return 4096
            self.calls.append((name, args[-1]))
            return ela.ATTN_OK

        return call


class Machine:
    def __init__(self, monkeypatch):
        self.current = types.SimpleNamespace(cuda_stream=10, device=DEVICE)
        self.made = []
        self.lib = Library()
        meta = torch.empty

        @contextlib.contextmanager
        def use(stream):
            before, self.current = self.current, stream
            yield
            self.current = before

        def empty(*shape, dtype=torch.float32, device=None, pin_memory=False):
            if device == "meta":
                return meta(*shape, dtype=dtype, device=device)
            shape = shape[0] if not isinstance(shape[0], int) else shape
            t = Tensor(shape, dtype, self.current)
            if device is not None:
                self.made.append(t)
            return t

        monkeypatch.setattr(ela, "load_library", lambda path=None: self.lib)
        monkeypatch.setattr(torch, "empty", empty)
        monkeypatch.setattr(torch, "empty_like", lambda t, **kw: empty(t.shape, dtype=t.dtype, device=t.device))
        monkeypatch.setattr(torch.cuda, "stream", use)
        monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.current)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: self.current.cuda_stream, raising=False)
        for cached in (ela._prefix_workspace_bytes, ela._bwd_workspace_bytes):
            cached.cache_clear()


@pytest.fixture
def machine(monkeypatch):
    yield Machine(monkeypatch)
    for cached in (ela._prefix_workspace_bytes, ela._bwd_workspace_bytes):
        cached.cache_clear()


def bf16(*shape):
    return Tensor(shape, torch.bfloat16)


def ready_args():
    return (bf16(2, 4, 6, 64), bf16(2, 2, 6, 64), Tensor((6,), torch.int32), Tensor((32,), torch.float64), bf16(64), bf16(64))


def ready(**kw):
    return ela.qk_norm_rope(*ready_args(), **kw)


def ready_bwd(**kw):
    return ela.qk_norm_rope_bwd(bf16(2, 4, 6, 64), bf16(2, 2, 6, 64), *ready_args(), **kw)


def prefix(**kw):
    return ela.attn_fwd_prefix(bf16(3, 8, 1, 64), bf16(2, 100, 64), bf16(2, 100, 64), bf16(3, 2, 20, 64), bf16(3, 2, 20, 64),
                               Tensor((3,), torch.int32), **kw)


def qkv(n=3, dtype=torch.bfloat16):
    return [Tensor((1, 2, 300, 128), dtype) for _ in range(n)]


def forward(**kw):
    return ela.attn_fwd(*qkv(), **kw)


def backward(**kw):
    return ela.attn_bwd(*qkv(4), Tensor((1, 2, 300), torch.float32), *qkv(1), **kw)


def forward_fp8(**kw):
    return ela.attn_fwd_fp8(*qkv(dtype=torch.uint8), (1.0, 1.0, 1.0), **kw)


def softmax(**kw):
    return ela.softmax_rows(bf16(4, 70000), **kw)


def layernorm(**kw):
    return ela.layernorm_rows(bf16(4, 64), bf16(64), bf16(64), **kw)


# the call, and how many buffers it allocates
CALLS = {"qk_norm_rope": (ready, 2), "qk_norm_rope_bwd": (ready_bwd, 5), "attn_fwd_prefix": (prefix, 3),
         "attn_fwd": (forward, 3), "attn_bwd": (backward, 4), "attn_fwd_fp8": (forward_fp8, 3), "softmax_rows": (softmax, 2),
         "layernorm_rows": (layernorm, 1)}


@pytest.mark.parametrize("name", CALLS)
def test_buffers_come_from_the_memory_of_the_stream_that_uses_them(machine, name):
    call, buffers = CALLS[name]
    side = types.SimpleNamespace(cuda_stream=20, device=DEVICE)
    caller = machine.current
    got = call(stream=side)
    got = [t for t in (got if isinstance(got, tuple) else (got,)) if t is not None]
    assert len(machine.made) == buffers
    assert all(t.made_on is side for t in machine.made)
    for t in machine.made:  # what is handed back may be freed while the caller's stream still reads it
        assert (caller in t.used_on) == any(t is g for g in got)
    assert [s for _, s in machine.lib.calls] == [20] and machine.current is caller
    # and without a stream: the current one's
    machine.made.clear()
    call()
    assert len(machine.made) == buffers and all(t.made_on is caller and not t.used_on for t in machine.made)
    assert machine.lib.calls[-1][1] == 10


def test_the_host_entry_takes_its_workspace_from_the_memory_of_the_stream(machine):
    side = types.SimpleNamespace(cuda_stream=20, device=DEVICE)
    ela.attn_fwd_host(*qkv(), out_h=bf16(1, 2, 300, 128), lse_h=Tensor((1, 2, 300), torch.float32), stream=side)
    assert [t.made_on for t in machine.made] == [side] and not machine.made[0].used_on


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(machine, name):
    call, _ = CALLS[name]
    with pytest.raises(ValueError):
        call(stream=types.SimpleNamespace(cuda_stream=20, device=torch.device("cuda", 1)))
    assert not machine.lib.calls


# ------------------------------------------------------------------ GPU
def _draw(seed, *shape):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def gpu_prefix(seed):
    R, Hq, Hk, d, P, C = 200, 8, 2, 128, 8192, 512
    a = [_draw(seed + i, *s) for i, s in enumerate([(R, Hq, 1, d), (Hk, P, d), (Hk, P, d), (R, Hk, C, d), (R, Hk, C, d)])]
    lens = torch.randint(1, C + 1, (R,), generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
    return lambda stream: ela.attn_fwd_prefix(*a, lens, stream=stream)


def gpu_ready_bwd(seed):
    B, H, N, d = 1, 16, 8192, 128
    g, gk, q, k = (_draw(seed + i, B, H, N, d) for i in range(4))
    wq, wk = _draw(seed + 4, d), _draw(seed + 5, d)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    inv = 10000.0 ** (-torch.arange(d // 2, dtype=torch.float64, device="cuda") / (d // 2))
    return lambda stream: ela.qk_norm_rope_bwd(g, gk, q, k, pos, inv, wq, wk, stream=stream)


def gpu_forward(seed):
    q, k, v = (_draw(seed + i, 1, 1, 16000, 128) for i in range(3))  # few units: the K/V split and its workspace
    return lambda stream: ela.attn_fwd(q, k, v, causal=True, stream=stream)


def gpu_fp8(seed):
    q, k, v = ((_draw(seed + i, 1, 4, 4096, 128).view(torch.uint8)[..., ::2] & 0x3f).contiguous() for i in range(3))
    return lambda stream: ela.attn_fwd_fp8(q, k, v, (0.1, 0.1, 0.1), stream=stream)


def gpu_softmax(seed):
    x = _draw(seed, 60, 300000)  # rows in segments, with a workspace
    return lambda stream: (ela.softmax_rows(x, stream=stream),)


GPU_CALLS = {"attn_fwd_prefix": gpu_prefix, "qk_norm_rope_bwd": gpu_ready_bwd, "attn_fwd": gpu_forward,
             "attn_fwd_fp8": gpu_fp8, "softmax_rows": gpu_softmax}


@gpu
@pytest.mark.parametrize("name", GPU_CALLS)
def test_calls_side_by_side_without_a_wait_give_the_serial_results(name):
    """Calls on the current stream, and at once one of the same sizes on another, whose buffers must not be theirs."""
    _build.build()
    one, two = GPU_CALLS[name](1), GPU_CALLS[name](100)
    want = one(None), two(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        a = [one(None) for _ in range(3)][-1]
        b = two(side)
        a2 = one(None)
        torch.cuda.synchronize()
        for got, w in ((a, want[0]), (b, want[1]), (a2, want[0])):
            assert all(torch.equal(x, y) for x, y in zip(got, w))
    assert ela.last_device_error() == ela.ATTN_OK


@gpu
def test_a_given_stream_inside_a_captured_graph():
    """A captured call on a stream that joined the capture: its buffers belong to the graph, as the current stream's do."""
    _build.build()
    calls = [make(1) for make in GPU_CALLS.values()]
    want = [call(None) for call in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = [(call(None), call(side), call(side)) for call in calls]
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for each, w in zip(got, want):
            for result in each:
                assert all(torch.equal(x, y) for x, y in zip(result, w))
    assert ela.last_device_error() == ela.ATTN_OK
