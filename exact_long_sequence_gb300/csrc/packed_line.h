// The line of work of attention over sequences of different lengths, as the
// kernels cut it: plain arithmetic, the same on the host and the device.
//
// The G query heads that share a key head are rows of one matrix: token t and
// head g of a sequence are row t G + g of its key head.  A query tile is the
// `tile_tokens` = 128 / G whole tokens that fit 128 rows, a block is two tiles.
// A unit is one block of a sequence at one key head against the keys that it
// sees.  On the line the units follow one another sequence by sequence, key
// head by key head, block by block; a unit is kUnitCost positions and one for each of its rows
// (query rows, pipeline fill, output), then one for each of its keys.  The line is cut into even
// stretches; a tile of 128 keys belongs to the
// stretch that holds the first position of it, so that every position is
// found from the lengths alone and the work of a stretch differs from the
// others' by a tile.
#pragma once

#include <cstdint>

#ifndef ELS_HD
#ifdef __CUDACC__
#define ELS_HD __host__ __device__ __forceinline__
#else
#define ELS_HD inline
#endif
#endif
// What a kernel needs a few times at its start is kept to one copy: fetching instructions is what that time is.
#ifdef __CUDACC__
#define ELS_HD_ONCE __host__ __device__ __noinline__
#else
#define ELS_HD_ONCE inline
#endif

namespace elsattn {

constexpr int kLineTile = 128;    // keys of a tile
// Start and end of a unit besides its rows' share.  With as many positions for every unit (and half for
// a key of a block of one tile) 24 prompts of 20 to 2000 tokens took 310 us (192 positions), 243 us
// (800) and 247 us (1100), 128 requests of one token 213, 224 and 236 us.
constexpr int kUnitCost = 200;
// A stretch is at least this long, so that each one between the first and the last of a unit has a tile of it.
constexpr int kLineLeast = 2 * kLineTile;

// a / b for a >= 0, b > 0: in 32 bits where both fit (a division in 64 costs a few hundred cycles).
static ELS_HD_ONCE int64_t line_div(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

// Positions of the first n blocks, all whole, of a sequence at one key head (LineSeq).
static ELS_HD_ONCE int64_t line_before(int nq, int nk, int block_tokens, int group, bool causal, int64_t n) {
    const int64_t unit = kUnitCost + block_tokens * group;
    if (!causal) return n * (unit + nk);
    // block i sees nk - nq + (i + 1) block_tokens keys, none where that is negative
    const int64_t off = static_cast<int64_t>(nk) - nq;
    int64_t i0 = off < 0 ? line_div(-off, block_tokens) : 0;
    if (i0 > n) i0 = n;
    return n * unit + (n - i0) * off + block_tokens * (n * (n + 1) / 2 - i0 * (i0 + 1) / 2);
}

// The units of one sequence at one key head.
struct LineSeq {
    int nq, nk;          // tokens, keys
    int tile_tokens;
    int group;           // query heads of the key head
    bool causal;         // token t sees the keys j <= t + nk - nq; otherwise all of them
    ELS_HD int block_tokens() const { return 2 * tile_tokens; }
    // (unsigned: the tokens rounded up to whole blocks may pass 2^31)
    ELS_HD int blocks() const {
        const unsigned bt = static_cast<unsigned>(block_tokens());
        return static_cast<int>((static_cast<unsigned>(nq) + bt - 1) / bt);
    }
    ELS_HD int tokens(int b) const {
        const int64_t left = nq - static_cast<int64_t>(b) * block_tokens();
        return left < block_tokens() ? static_cast<int>(left) : block_tokens();
    }
    // Keys that token t sees.
    ELS_HD int sees(int64_t t) const {
        if (!causal) return nk;
        const int64_t v = t + 1 + nk - nq;
        return v < 0 ? 0 : v > nk ? nk : static_cast<int>(v);
    }
    // Keys that a block sees: those of its last token.
    ELS_HD int keys(int b) const { return sees(static_cast<int64_t>(b) * block_tokens() + tokens(b) - 1); }
    ELS_HD int unit_cost(int b) const { return kUnitCost + tokens(b) * group; }
    // Positions of the blocks before b (b < blocks(), so all of them are whole).
    ELS_HD int64_t before(int b) const { return line_before(nq, nk, block_tokens(), group, causal, b); }
    ELS_HD int64_t cost(int b) const { return static_cast<int64_t>(unit_cost(b)) + keys(b); }
    // All blocks.
    ELS_HD int64_t length() const {
        if (nq <= 0) return 0;
        const int last = blocks() - 1;
        return before(last) + cost(last);
    }
};

// The line of the gradient: a unit is a tile of 128 keys of a sequence at one key
// head with the tokens that see one of them, which are the last ones; its query
// blocks of `block_tokens` = 64 / G tokens begin at the first of those.  A unit is
// kKeyUnitBlocks blocks and then its tokens, one position each (24 texts of 10 to 2501 tokens, 24 heads of 4, with 2, 4,
// 7, 10 and 14 blocks: 812, 793, 767, 779 and 791 us).
constexpr int kKeyUnitBlocks = 7;
constexpr int kKeyLineLeast = 8;   // blocks of the shortest stretch
static ELS_HD_ONCE int64_t line_tiles_before(int nq, int nk, int unit_cost, bool causal, int64_t n) {
    const int64_t off = static_cast<int64_t>(nk) - nq;
    if (!causal || nq == 0) return n * (unit_cost + static_cast<int64_t>(nq));
    // tile i has all tokens while 128 i <= nk - nq, then nk - 128 i of them
    int64_t i0 = off < 0 ? 0 : off / kLineTile + 1;
    if (i0 > n) i0 = n;
    return n * unit_cost + i0 * nq + (n - i0) * nk - kLineTile * (n * (n - 1) / 2 - i0 * (i0 - 1) / 2);
}
struct LineKeys {
    int nq, nk;          // tokens, keys
    int block_tokens;
    bool causal;
    ELS_HD int tiles() const { return static_cast<int>((static_cast<unsigned>(nk) + kLineTile - 1) / kLineTile); }
    ELS_HD int unit_cost() const { return kKeyUnitBlocks * block_tokens; }
    // The first token that sees a key of tile j (of tokens that there are, since the last one sees all keys).
    ELS_HD int first(int j) const {
        if (!causal) return 0;
        const int64_t t = static_cast<int64_t>(j) * kLineTile - (static_cast<int64_t>(nk) - nq);
        return t < 0 || nq == 0 ? 0 : static_cast<int>(t);
    }
    ELS_HD int64_t cost(int j) const { return unit_cost() + nq - first(j); }
    // Positions of the tiles before j.
    ELS_HD int64_t before(int j) const { return line_tiles_before(nq, nk, unit_cost(), causal, j); }
    ELS_HD int64_t length() const { return before(tiles()); }
};

// What a stretch [x0, x1) has of a unit whose tiles (or blocks) begin at `first` and every `step` positions after it.
struct LinePart {
    int t0, t1;     // its tiles [t0, t1)
    ELS_HD LinePart(int64_t first, int tiles, int step, int64_t x0, int64_t x1) {
        const int64_t a = x0 > first ? line_div(x0 - first + step - 1, step) : 0;
        const int64_t b = x1 > first ? line_div(x1 - first + step - 1, step) : 0;
        t0 = a < tiles ? static_cast<int>(a) : tiles;
        t1 = b < tiles ? static_cast<int>(b) : tiles;
    }
};

// Length of the stretches that a line of `total` is cut into, `most` of them at most.
ELS_HD int64_t line_stretch(int64_t total, int most, int least = kLineLeast) {
    const int64_t even = line_div(total + most - 1, most);
    return even < least ? least : even;
}

// Whether units of up to most_keys keys and most_rows rows a block are left whole on stretches of `len`, each at one stretch.
// A cut costs pieces of its rows and their merge, a whole unit the wait for whoever has the longest: whole with up to
// ten keys a row, and two and a half stretches to a unit.  Cut and whole, us (causal, 32 heads of 8 unless said, replayed from a
// graph): 24 prompts of 20 to 2000 tokens 223 and 204 (210 and 199 in the order of their lengths), 1200 tokens 40 and 28, 2400
// tokens at 16 heads of 4 51 and 40, 8 of 600 without the mask 73 and 62; but 4 prompts of 100 to 4000 tokens 157 and 163, one of
// 4800 164 and 175, 7 clips of 500 to 6143 at 16 heads, d = 64, 372 and 406, 128 requests of one token 184 and 204.
constexpr int kWholeRowKeys = 10;
ELS_HD bool line_whole(int most_keys, int most_rows, int64_t len) {
    return most_keys <= kWholeRowKeys * most_rows && 2 * (static_cast<int64_t>(kUnitCost) + most_rows + most_keys) <= 5 * len;
}

}  // namespace elsattn
