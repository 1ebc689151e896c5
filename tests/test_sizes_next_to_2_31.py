"""Sizes next to 2^31 of the shared-prefix attention and the preparation are refused: the kernels round
them up to whole tiles, blocks and steps in 32 bits.  (Overlapping views make such a call possible.)"""
import pytest

import exact_long_sequence_gb300 as ela

import test_prefix as prefix_tests
import test_qk_norm_rope as ready_tests
from test_prefix import lib  # noqa: F401

TOP = 2 ** 31 - 1


@pytest.mark.parametrize("over", [
    dict(P=TOP, C=0, Hk=1, Hq=1, R=1, kps=(8, 8), vps=(8, 8)), dict(P=TOP - 200, C=0, Hk=1, Hq=1, R=1, kps=(8, 8), vps=(8, 8)),
    dict(P=0, C=TOP, Hk=1, Hq=1, R=1, kos=(8, 8, 8), vos=(8, 8, 8)), dict(P=10, C=TOP, Hk=1, Hq=1, R=1, kos=(8, 8, 8), vos=(8, 8, 8)),
    dict(P=10, C=0, Hk=1, Hq=1, R=1, T=TOP, qs=(8, 8, 8), os=(8, 8, 8)), dict(P=10, C=0, Hk=1, Hq=1, R=TOP, qs=(8, 8, 8), os=(8, 8, 8)),
])
def test_prefix(lib, over):  # noqa: F811
    assert prefix_tests.cdll_call(lib, **over) == ela.ATTN_ERR_INVALID_ARG
    shape = {**dict(R=3, Hq=8, Hk=2, T=1, P=100, C=50, d=64), **{k: v for k, v in over.items() if isinstance(v, int)}}
    assert lib.attn_fwd_prefix_workspace_bytes(*[shape[k] for k in ("R", "Hq", "Hk", "T", "P", "C", "d")]) == 0


@pytest.mark.parametrize("fn", ["fwd", "bwd"])
@pytest.mark.parametrize("over", [dict(B=1, N=1, Hq=TOP), dict(B=1, N=1, Hk=TOP), dict(B=1, N=TOP, Hq=1, Hk=1), dict(B=TOP, N=1, Hq=1, Hk=1)])
def test_preparation(lib, fn, over):  # noqa: F811
    assert ready_tests.cdll_call(lib, fn, **over) == ela.ATTN_ERR_INVALID_ARG
