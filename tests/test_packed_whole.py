"""Calls whose units are left whole (line_whole of packed_line.h) and calls next to the rule's bounds, against the definition."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_long_sequence_gb300", "csrc")
PROGRAM = r"""
#include "packed_line.h"
using namespace elsattn;
extern "C" {
int whole(int keys, int rows, int64_t len) { return line_whole(keys, rows, len); }
int64_t length(int nq, int nk, int tt, int g, int causal) { return LineSeq{nq, nk, tt, g, causal != 0}.length(); }
int64_t cost(int nq, int nk, int tt, int g, int causal, int b) { return LineSeq{nq, nk, tt, g, causal != 0}.cost(b); }
int blocks(int nq, int nk, int tt, int g, int causal) { return LineSeq{nq, nk, tt, g, causal != 0}.blocks(); }
int64_t stretch(int64_t total, int most) { return line_stretch(total, most); }
}
"""


@pytest.fixture(scope="module")
def line(tmp_path_factory):
    at = tmp_path_factory.mktemp("whole")
    src, so = at / "whole.cpp", at / "whole.so"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.whole.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int64]
    lib.stretch.argtypes = [ctypes.c_int64, ctypes.c_int]
    for f in ("length", "cost", "stretch"):
        getattr(lib, f).restype = ctypes.c_int64
    return lib


def test_bounds(line):
    assert line.whole(0, 0, 256)
    assert line.whole(2560, 256, 1 << 40) and not line.whole(2561, 256, 1 << 40)
    assert line.whole(40, 4, 1 << 40) and not line.whole(41, 4, 1 << 40)  # few rows: a merge of them is cheap
    assert not line.whole((1 << 31) - 1, 256, 1 << 60)
    longest = 200 + 256 + 1144
    assert line.whole(1144, 256, longest * 2 // 5) and not line.whole(1144, 256, longest * 2 // 5 - 1)


def loads(line, seqs, Hk, g, causal, most):
    """Positions of the units whose middle lies in each stretch, and the longest unit."""
    tt = 128 // g
    total = sum(Hk * line.length(nq, nk, tt, g, causal) for nq, nk in seqs)
    size = line.stretch(total, most)
    at, load, longest = 0, [0] * most, 0
    for nq, nk in seqs:
        for _ in range(Hk):
            for b in range(line.blocks(nq, nk, tt, g, causal)):
                c = line.cost(nq, nk, tt, g, causal, b)
                load[(at + c // 2) // size] += c
                at, longest = at + c, max(longest, c)
    return load, size, longest


def test_loads(line):
    """Every unit is one stretch's, and no stretch has more than its length and the longest unit."""
    rng = random.Random(5)
    for _ in range(100):
        seqs = [(rng.randrange(1, 900), rng.randrange(0, 2500)) for _ in range(rng.randrange(1, 9))]
        load, size, longest = loads(line, seqs, rng.choice([1, 4, 8]), rng.choice([1, 2, 3, 64]), rng.random() < 0.5, 152)
        assert max(load) <= size + longest
    # as many equal units as stretches: one each, although the last of each head is a little shorter
    load, _, longest = loads(line, [(1200, 1200)], 8, 4, False, 152)
    assert max(load) == longest


@pytest.mark.gpu
@pytest.mark.parametrize("ql,kl,Hq,Hk,d,causal", [
    ([1200], None, 32, 8, 128, False),                            # one unit to a stretch
    ([1200], None, 16, 16, 128, True),                            # fewer units than stretches
    ([300] * 8, None, 32, 8, 128, True),
    ([300, 1, 0, 900, 64, 257] * 4, None, 24, 8, 64, True),       # (three heads: 126 rows a tile)
    ([255, 256, 1, 0, 300] * 9, [700, 2, 900, 40, 0] * 9, 8, 8, 128, True),   # also rows that see nothing, and queries without keys
    ([255, 256, 1, 0, 300] * 9, [700, 2, 900, 40, 0] * 9, 8, 8, 64, False),
    ([300] * 40, [2560] * 40, 2, 2, 64, True),                    # the most keys of the rule, and one more
    ([300] * 40, [2561] * 40, 2, 2, 64, True),
    ([1] * 700, [40] * 700, 8, 2, 128, True),                     # the most keys of single tokens, and one more
    ([1] * 700, [40] * 699 + [41], 8, 2, 128, False),
    ([200] * 300, None, 2, 2, 64, True),                          # more sequences than lanes
])
def test_against_the_definition(ql, kl, Hq, Hk, d, causal):
    from test_packed import run
    run(ql, kl, Hq=Hq, Hk=Hk, d=d, causal=causal, seed=len(ql))


@pytest.mark.gpu
def test_a_graph_whose_lengths_change_sides():
    """The rule is the device's: a captured call replayed with lengths on either side of it."""
    import torch

    import exact_long_sequence_gb300 as ela
    from packed_ref import check, packed
    n, d = 4096, 64
    g = torch.Generator("cuda").manual_seed(3)
    q, k, v = (torch.randn((8, n, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    starts = torch.zeros(9, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((8, n), device="cuda")
    work = torch.empty(ela.packed_workspace_bytes(8, n, n, 8, 8, d), dtype=torch.uint8, device="cuda")
    ela.attn_fwd_packed(q, k, v, starts, causal=True, out=out, lse=lse, workspace=work)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ela.attn_fwd_packed(q, k, v, starts, causal=True, out=out, lse=lse, workspace=work)
    for cuts in ([512 * i for i in range(9)], [0, 4096] + [4096] * 7, [0, 3000, 3001, 3100, 3600, 3600, 3700, 4000, 4096],
                 [500 * i for i in range(9)], [0] * 8 + [3900]):
        starts.copy_(torch.tensor(cuts, dtype=torch.int32))
        out.fill_(7)
        lse.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert ela.last_device_error() == ela.ATTN_OK
        check(out, lse, packed(q, k, v, cuts, cuts, True, ela.default_scale(d)))
        assert bool((out[:, cuts[-1]:] == 7).all()) and bool((lse[:, cuts[-1]:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
def test_several_turns(causal):
    """As many bytes as give each CTA two stretches of the forward's line (above 128 MB of K and V) and three of the gradient's
    (above 300 MB of Q, dO and dQ's sums), cut units among them."""
    import torch

    from test_packed import run
    from test_packed_bwd import run as run_bwd
    lens = torch.randint(0, 121, (150,), generator=torch.Generator().manual_seed(1)).tolist()
    lens[70] = 3100
    run(lens, Hq=32, Hk=32, d=128, causal=causal, seed=1)
    run_bwd(lens, Hq=32, Hk=32, d=128, causal=causal, seed=2)
