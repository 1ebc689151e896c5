"""The abort path of the packed and paged kernels, driven on the GPU without a fault, as test_abort.py does for the forward's.

attn_debug_arm_timeout arms a one-shot for the next call: a short wait limit, and each even CTA arms the barrier of its
first query copy without the copy.  The product warp's wait on it runs out; the CTA's other roles leave their loops at
their next wait, copies, products and reductions in flight are waited for, and tensor memory is freed.  The CTAs beside it
end as usual, and the merging kernels read cuts of both.  Each case checks that the status comes back, well before the default
limit, and that the next call, not armed, gives what a call before gave.
"""
import time

import pytest
import torch

import exact_long_sequence_gb300 as ela
from test_packed_streams import CALLS, draw, lengths, same

pytestmark = pytest.mark.gpu
LIMIT_NS = 20_000_000


def whole(seed):
    """Units that are left whole by their lengths, two query tiles each."""
    st, N = lengths(seed, 40, 300)
    q, k, v = draw(seed, 8, N, 64), draw(seed + 1, 8, N, 64), draw(seed + 2, 8, N, 64)
    return lambda: ela.attn_fwd_packed(q, k, v, st, causal=True)


def short_gradient(seed):
    """Up to eight blocks of tokens: no unit of the gradient is cut."""
    st = torch.tensor([0, 100, 101, 300], dtype=torch.int32, device="cuda")
    q, k, v, do = draw(seed, 32, 300, 64), draw(seed + 1, 32, 300, 64), draw(seed + 2, 32, 300, 64), draw(seed + 3, 32, 300, 64)
    o, lse = ela.attn_fwd_packed(q, k, v, st, causal=True)
    return lambda: ela.attn_bwd_packed(q, k, v, o, lse, do, st, causal=True)


@pytest.mark.parametrize("name", [*CALLS, "whole", "short gradient"])
def test_abort_reports_timeout_and_the_next_call_is_as_before(name):
    call = {"whole": whole, "short gradient": short_gradient, **CALLS}[name](5)
    want = call()
    assert ela.last_device_error() == ela.ATTN_OK
    assert ela.debug_arm_timeout(LIMIT_NS) == ela.ATTN_OK
    t0 = time.perf_counter()
    call()
    status = ela.last_device_error()
    elapsed = time.perf_counter() - t0
    assert status == ela.ATTN_ERR_TIMEOUT, status
    assert elapsed < 1.5, elapsed
    for _ in range(2):
        got = call()
        assert ela.last_device_error() == ela.ATTN_OK
        same(got, want)
