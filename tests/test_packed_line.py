"""The line of work of attention over lengths (packed_line.h), compiled for the host: closed sums against plain ones, and
every tile of every unit in exactly one stretch."""
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
int blocks(int nq, int nk, int tt, int causal) { return LineSeq{nq, nk, tt, causal != 0}.blocks(); }
int keys(int nq, int nk, int tt, int causal, int b) { return LineSeq{nq, nk, tt, causal != 0}.keys(b); }
int weight(int nq, int nk, int tt, int causal, int b) { return LineSeq{nq, nk, tt, causal != 0}.weight(b); }
int64_t before(int nq, int nk, int tt, int causal, int b) { return LineSeq{nq, nk, tt, causal != 0}.before(b); }
int64_t length(int nq, int nk, int tt, int causal) { return LineSeq{nq, nk, tt, causal != 0}.length(); }
int64_t stretch(int64_t total, int most) { return line_stretch(total, most); }
void part(int64_t start, int tiles, int weight, int64_t x0, int64_t x1, int* out) {
    const LinePart p(start, tiles, weight, x0, x1);
    out[0] = p.t0;
    out[1] = p.t1;
}
int unit_cost() { return kUnitCost; }
}
"""


@pytest.fixture(scope="module")
def line(tmp_path_factory):
    at = tmp_path_factory.mktemp("line")
    src, so = at / "line.cpp", at / "line.so"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    for f in ("before", "length", "stretch"):
        getattr(lib, f).restype = ctypes.c_int64
    lib.stretch.argtypes = [ctypes.c_int64, ctypes.c_int]
    lib.part.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.POINTER(ctypes.c_int)]
    return lib


def plain_keys(nq, nk, tt, causal, b):
    last = min(nq, (b + 1) * 2 * tt) - 1
    return max(0, min(nk, last + 1 + nk - nq)) if causal else nk


def test_sums(line):
    rng = random.Random(0)
    for _ in range(3000):
        nq, nk = rng.choice([0, 1, 5, rng.randrange(3000)]), rng.choice([0, 1, rng.randrange(3000)])
        tt, causal = rng.choice([128, 64, 42, 25, 2]), rng.random() < 0.7
        nb = line.blocks(nq, nk, tt, causal)
        assert nb == -(-nq // (2 * tt))
        at = 0
        for b in range(nb):
            assert line.before(nq, nk, tt, causal, b) == at
            keys = line.keys(nq, nk, tt, causal, b)
            assert keys == plain_keys(nq, nk, tt, causal, b)
            w = line.weight(nq, nk, tt, causal, b)
            assert w == (2 if min(nq - b * 2 * tt, 2 * tt) > tt else 1)
            at += line.unit_cost() + w * keys
        assert line.length(nq, nk, tt, causal) == at


def test_sums_next_to_32_bits(line):
    n = (1 << 31) - 513
    for nq, nk, tt in ((n, n, 128), (n, 1, 2), (1, n, 128), (n, n // 2, 128)):
        nb = line.blocks(nq, nk, tt, 1)
        assert nb == -(-nq // (2 * tt))
        assert line.keys(nq, nk, tt, 1, nb - 1) == nk
        assert line.keys(nq, nk, tt, 1, 0) == plain_keys(nq, nk, tt, True, 0)
        off = nk - nq
        full = nb - 1
        plain = full * line.unit_cost()
        i0 = min(full, -off // (2 * tt)) if off < 0 else 0
        plain += 2 * ((full - i0) * off + 2 * tt * (full * (full + 1) // 2 - i0 * (i0 + 1) // 2))
        assert line.before(nq, nk, tt, 1, full) == plain


def test_every_tile_is_in_one_stretch(line):
    rng = random.Random(1)
    out = (ctypes.c_int * 2)()
    for _ in range(300):
        tt, causal, Hk = rng.choice([128, 64, 42, 2]), rng.random() < 0.7, rng.choice([1, 2, 3])
        seqs = [(rng.choice([0, 1, 3, 200, rng.randrange(1500)]), rng.choice([0, 1, 128, rng.randrange(4000)]))
                for _ in range(rng.randrange(1, 8))]
        total = sum(Hk * line.length(nq, nk, tt, causal) for nq, nk in seqs)
        most = rng.choice([1, 4, 152])
        size = line.stretch(total, most)
        assert size * most >= total and size >= 256
        start = 0
        for nq, nk in seqs:
            for _h in range(Hk):
                for b in range(line.blocks(nq, nk, tt, causal)):
                    keys, w = line.keys(nq, nk, tt, causal, b), line.weight(nq, nk, tt, causal, b)
                    tiles = -(-keys // 128)
                    got, pieces = 0, []
                    for i in range(most):
                        line.part(start, tiles, w, i * size, min((i + 1) * size, total), out)
                        if out[0] < out[1]:
                            assert out[0] == got
                            got = out[1]
                            pieces.append(i)
                    assert got == tiles
                    if tiles:  # the pieces' count as the kernel leaves it for the one that merges them
                        assert pieces == list(range(pieces[0], pieces[-1] + 1))
                        last = (start + line.unit_cost() + (tiles - 1) * 128 * w) // size
                        assert last == pieces[-1]
                    start += line.unit_cost() + w * keys
        assert start == total
