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
int blocks(int nq, int nk, int tt, int g, int causal) { return LineSeq{nq, nk, tt, g, causal != 0}.blocks(); }
int keys(int nq, int nk, int tt, int g, int causal, int b) { return LineSeq{nq, nk, tt, g, causal != 0}.keys(b); }
int unit(int nq, int nk, int tt, int g, int causal, int b) { return LineSeq{nq, nk, tt, g, causal != 0}.unit_cost(b); }
int64_t before(int nq, int nk, int tt, int g, int causal, int b) { return LineSeq{nq, nk, tt, g, causal != 0}.before(b); }
int64_t length(int nq, int nk, int tt, int g, int causal) { return LineSeq{nq, nk, tt, g, causal != 0}.length(); }
int k_tiles(int nq, int nk, int bt, int causal) { return LineKeys{nq, nk, bt, causal != 0}.tiles(); }
int k_first(int nq, int nk, int bt, int causal, int j) { return LineKeys{nq, nk, bt, causal != 0}.first(j); }
int k_unit(int nq, int nk, int bt, int causal) { return LineKeys{nq, nk, bt, causal != 0}.unit_cost(); }
int64_t k_cost(int nq, int nk, int bt, int causal, int j) { return LineKeys{nq, nk, bt, causal != 0}.cost(j); }
int64_t k_before(int nq, int nk, int bt, int causal, int j) { return LineKeys{nq, nk, bt, causal != 0}.before(j); }
int64_t k_length(int nq, int nk, int bt, int causal) { return LineKeys{nq, nk, bt, causal != 0}.length(); }
int64_t stretch(int64_t total, int most) { return line_stretch(total, most); }
int64_t k_stretch(int64_t total, int most, int bt) { return line_stretch(total, most, kKeyLineLeast * bt); }
void part(int64_t first, int tiles, int step, int64_t x0, int64_t x1, int* out) {
    const LinePart p(first, tiles, step, x0, x1);
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
    for f in ("before", "length", "stretch", "k_cost", "k_before", "k_length", "k_stretch"):
        getattr(lib, f).restype = ctypes.c_int64
    lib.stretch.argtypes = [ctypes.c_int64, ctypes.c_int]
    lib.k_stretch.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int]
    lib.part.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.POINTER(ctypes.c_int)]
    return lib


def plain_keys(nq, nk, tt, causal, b):
    last = min(nq, (b + 1) * 2 * tt) - 1
    return max(0, min(nk, last + 1 + nk - nq)) if causal else nk


def test_sums(line):
    rng = random.Random(0)
    for _ in range(3000):
        nq, nk = rng.choice([0, 1, 5, rng.randrange(3000)]), rng.choice([0, 1, rng.randrange(3000)])
        g, causal = rng.choice([1, 2, 3, 5, 64]), rng.random() < 0.7
        tt = 128 // g
        nb = line.blocks(nq, nk, tt, g, causal)
        assert nb == -(-nq // (2 * tt))
        at = 0
        for b in range(nb):
            assert line.before(nq, nk, tt, g, causal, b) == at
            keys = line.keys(nq, nk, tt, g, causal, b)
            assert keys == plain_keys(nq, nk, tt, causal, b)
            unit = line.unit(nq, nk, tt, g, causal, b)
            assert unit == line.unit_cost() + min(nq - b * 2 * tt, 2 * tt) * g
            at += unit + keys
        assert line.length(nq, nk, tt, g, causal) == at


def test_sums_next_to_32_bits(line):
    n = (1 << 31) - 513
    for nq, nk, tt in ((n, n, 128), (n, 1, 2), (1, n, 128), (n, n // 2, 128)):
        g = 128 // tt
        nb = line.blocks(nq, nk, tt, g, 1)
        assert nb == -(-nq // (2 * tt))
        assert line.keys(nq, nk, tt, g, 1, nb - 1) == nk
        assert line.keys(nq, nk, tt, g, 1, 0) == plain_keys(nq, nk, tt, True, 0)
        off = nk - nq
        full = nb - 1
        plain = full * (line.unit_cost() + 2 * tt * g)
        i0 = min(full, -off // (2 * tt)) if off < 0 else 0
        plain += (full - i0) * off + 2 * tt * (full * (full + 1) // 2 - i0 * (i0 + 1) // 2)
        assert line.before(nq, nk, tt, g, 1, full) == plain


def cover(line, size, most, total, units):
    """Every tile of every unit (first position, tiles, step, end) lies in one stretch, and the pieces are neighbours whose
    count is what the kernels leave for the one that merges them."""
    out = (ctypes.c_int * 2)()
    for first, tiles, step in units:
        got, pieces = 0, []
        for i in range(max(0, first // size - 1), min(most, (first + tiles * step) // size + 2)):
            line.part(first, tiles, step, i * size, min((i + 1) * size, total), out)
            if out[0] < out[1]:
                assert out[0] == got
                got = out[1]
                pieces.append(i)
        assert got == tiles
        if tiles:
            assert pieces == list(range(pieces[0], pieces[-1] + 1))
            assert (first + (tiles - 1) * step) // size == pieces[-1]


def test_every_tile_is_in_one_stretch(line):
    rng = random.Random(1)
    for _ in range(300):
        g, causal, Hk = rng.choice([1, 2, 3, 64]), rng.random() < 0.7, rng.choice([1, 2, 3])
        tt = 128 // g
        seqs = [(rng.choice([0, 1, 3, 200, rng.randrange(1500)]), rng.choice([0, 1, 128, rng.randrange(4000)]))
                for _ in range(rng.randrange(1, 8))]
        total = sum(Hk * line.length(nq, nk, tt, g, causal) for nq, nk in seqs)
        most = rng.choice([1, 4, 152])
        size = line.stretch(total, most)
        assert size * most >= total and size >= 128
        start, units = 0, []
        for nq, nk in seqs:
            for _h in range(Hk):
                for b in range(line.blocks(nq, nk, tt, g, causal)):
                    keys, unit = line.keys(nq, nk, tt, g, causal, b), line.unit(nq, nk, tt, g, causal, b)
                    units.append((start + unit, -(-keys // 128), 128))
                    start += unit + keys
        assert start == total
        cover(line, size, most, total, units)


def test_lines_of_the_gradient(line):
    rng = random.Random(2)
    for _ in range(400):
        bt, causal, Hk = rng.choice([64, 32, 21, 9, 1]), rng.random() < 0.7, rng.choice([1, 2, 3])
        seqs = [(rng.choice([0, 1, 3, 200, rng.randrange(900)]), rng.choice([0, 1, 128, rng.randrange(3000)]))
                for _ in range(rng.randrange(1, 6))]
        start, units = 0, []
        for nq, nk in seqs:
            for _h in range(Hk):
                at = 0
                tiles = line.k_tiles(nq, nk, bt, causal)
                assert tiles == -(-nk // 128)
                for j in range(tiles):
                    # the first token that sees the tile's first key: none before it, and all from it on
                    sees = [t for t in range(nq) if not causal or j * 128 <= t + nk - nq]
                    assert nq - line.k_first(nq, nk, bt, causal, j) == len(sees)
                    assert line.k_before(nq, nk, bt, causal, j) == at
                    assert line.k_cost(nq, nk, bt, causal, j) == line.k_unit(nq, nk, bt, causal) + len(sees)
                    units.append((start + at + line.k_unit(nq, nk, bt, causal), -(-len(sees) // bt), bt))
                    at += line.k_unit(nq, nk, bt, causal) + len(sees)
                assert line.k_length(nq, nk, bt, causal) == at
                start += at
        most = rng.choice([1, 4, 152])
        size = line.k_stretch(start, most, bt)
        assert size * most >= start and size >= bt
        cover(line, size, most, start, units)
