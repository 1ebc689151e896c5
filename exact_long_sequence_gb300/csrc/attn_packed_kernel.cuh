// Attention over sequences of different lengths, for sm_103a, in two forms:
//   packed: the tokens of all sequences follow one another in Q, K and V, and a
//     sequence's queries see its own keys (all, or causally);
//   paged (PAGED): T new tokens of each of R requests, whose keys and values
//     lie in pages of a cache; the new tokens see the keys before them and, of
//     one another, what a mask allows (a tree of drafted tokens).
// With n_s queries and m_s keys of sequence s, and G query heads to a key head,
//     O_i = sum_j p_ij V_j,  p_ij = exp(scale q_i . k_j - LSE_i) over the keys that i sees.
//
// The rows of a key head are its tokens' heads, row = token G + head: a tile of
// 128 rows is 128 / G tokens, whose K/V are read once for all G heads, and a
// causal tile crosses the diagonal in 128 / G keys instead of 128.
//
// Work is laid on a line (packed_line.h) and cut into even stretches, so that
// all SMs end together whatever the lengths are; the lengths are device data,
// and each CTA works out its own stretches from them.  A unit (block of rows at
// a key head) inside one stretch is written by its CTA; the pieces of a unit
// that stretches cut are left in fp32 and merged by attn_packed_combine_kernel,
//     LSE = log sum_s exp(LSE_s),  O = sum_s exp(LSE_s - LSE) O_s,
// the combination step of the online softmax.  Where all K and V together would
// not stay in L2, the line has several stretches a CTA, run in the order of the
// line, so that all CTAs are in one part of it at a time.
//
// Roles and pipeline are those of attn_prefix_kernel: two chains (S_c, O_c in
// TMEM, softmax warpgroup c) alternate, so that the tensor core works on one
// while the softmax of the other runs.  An item (a stretch's part of a unit) of
// more than one query tile has a tile on each chain, and both share the K/V
// tiles; an item of one query tile gives the chains its K/V tiles in turn.
//   warp 0  TMA producer of K_j, V_j into a ring of stages
//   warp 1  tcgen05.mma issuer; owns the TMEM allocation
//   warp 2  scheduler: the CTA's items, through a ring of descriptions
//   warp 3  Q loader
//   warps 4-7, 8-11  softmax warpgroups
//   warps 12-15      epilogue: O from TMEM to memory.  While they write an item's O the softmax warps are at
//     the next item's first tiles, which is what short sequences are made of.
//
// Measured, with 32 heads of 8, d = 128: documents of 3001 to 16384 tokens, causal, 2.19 ms, 1.41 PFLOP/s (the chain
// of score product, softmax and output product; tensor pipe 66 % active); 24 prompts of 20 to 2000 tokens 214 to 229 us, 740 to
// 793 TFLOP/s (the ends of items, whose instructions come from far, and whole units of unequal size: tensor pipe 37 %); paged,
// single tokens of 128 requests on up to 4099 keys 186 us, 5.8 TB/s, and trees of 24 drafts of 48 requests on up to 9001
// 170 us, 5.9 TB/s (HBM).
//
// Bytes that a thread spills and reads back, at its 128 registers: packed 20 and 40 (d = 128), 16 and 32 (64); paged 12 and 28
// (d = 128), 164 and 356 (64).
#pragma once

#include <cuda.h>
#include <cstddef>
#include <cstdint>
#include <type_traits>

#include "attn_prefix_kernel.cuh"
#include "packed_line.h"

namespace elsattn {

constexpr int kPkTailBox = 32;     // keys per TMA box of a tile that is not full
constexpr int kPkMostGroup = 64;   // most query heads of a key head
constexpr int kPkThreads = 512;
constexpr int kPkReaders = 15;     // of an item: producer, MMA, Q loader, eight softmax and four epilogue warps

struct PackedParams {
    // packed: [R + 1] first tokens of the sequences in Q, and in K and V (each clipped to the tensors)
    const int32_t* q_starts;
    const int32_t* k_starts;
    // paged: [R] keys of the requests, the new tokens among them (negative: padding), and their pages
    const int32_t* lens;
    const int32_t* table;      // request r's i-th page at r * table_stride + i
    const uint32_t* mask;      // [R, T, words] bits: new token t sees new token j; nullptr: those up to itself
    int64_t table_stride;
    int words;                 // 32-bit words of a mask row
    int page_log2, box;        // keys of a page; rows of a TMA box of it (at most 128)
    int pages;                 // of the cache
    int cap;                   // most keys of a request: the table's pages
    int R, Hk, G, T;           // T: paged only
    int Nq, Nk;                // packed: tokens and keys of the tensors
    int tile_tokens, qrows;    // of a query tile: whole tokens, and rows
    int orows;                 // partial rows kept for a piece
    bool causal;               // token t sees the keys j <= t + nk - nq
    int stretches;             // how many stretches the line has at most (a multiple of the grid)
    bool whole;                // no unit is cut, whatever the lengths are: each is in the stretch that its middle is in
    __nv_bfloat16* o;
    int64_t os[3];             // strides in elements: request (paged), head, token
    float* lse;
    int64_t ls[2];             // request (paged), head
    float* part_o;             // [2 stretches][orows][d]: slot 2 i + 1 is the piece that begins a unit in stretch i, 2 i one that goes on
    float* part_lse;           // [2 stretches][orows]
    struct PackedCut* cuts;    // [stretches]
    uint32_t* error_word;
    uint64_t timeout_ns;
    float scale_log2, max_scale_log2;
    uint32_t negate_scores;
    uint32_t withhold_first_q; // test hook: not 0 makes each even CTA arm its first query tile's barrier without the copy
};

// The unit whose pieces begin in a stretch (pieces: 0 where none is cut there).
struct PackedCut {
    int pieces;
    int head, req, tok0, nrows;
    int pad[3];
};

struct PackedItem {
    int ntiles;      // of K/V in this part of the unit; -1: no more items; 0: the unit sees no key
    int tile0;       // the first of them
    int ntiles0;     // how many of them its first query tile takes
    int klen;        // keys of the sequence that the unit sees
    int k0;          // packed: the sequence's first key
    int req;         // paged: the request
    int head;        // key head
    int tok0;        // first token of the block, in the tensor (packed) or the request
    int nrows;       // rows of the block
    int sees0;       // keys that the block's first token sees (can be negative: none)
    int step;        // ... and how many more each next token: 1 or 0
    int slot;        // partial slot; -1: the unit is whole
};
static_assert(sizeof(PackedItem) == 48, "read by words");

template <int D>
struct PackedSmem {
    static constexpr int kTile = tile_bytes(D);
    static constexpr int kStages = kv_stages_for(D);
    static constexpr int kQOff = 0;
    static constexpr int kRingOff = kQTiles * kTile;
    // weights of the rows' O for the epilogue: [2][128] by tile; of an item on both chains [128] pairs, where
    // chain 1 leaves its (m, l) first
    static constexpr int kWeightOff = kRingOff + kStages * kTile;
    static constexpr int kItemOff = kWeightOff + 128 * 8;
    static constexpr int kBarOff = kItemOff + kPfxItemRing * static_cast<int>(sizeof(PackedItem));
    static constexpr int kKvFull = 0;
    static constexpr int kKvEmpty = kKvFull + kStages;
    static constexpr int kQFull = kKvEmpty + kStages;     // [2] by slot
    static constexpr int kQEmpty = kQFull + 2;            // [2]
    static constexpr int kSFull = kQEmpty + 2;            // [2] by chain, as all below
    static constexpr int kPHalf = kSFull + 2;             // [2] first half of P stored, O rescaled
    static constexpr int kPFull = kPHalf + 2;             // [2]
    static constexpr int kOFull = kPFull + 2;             // [2]
    static constexpr int kOEmpty = kOFull + 2;            // [2]
    static constexpr int kWFull = kOEmpty + 2;            // [2] the chain's weights are there (of an item on both: chain 0's)
    static constexpr int kWEmpty = kWFull + 2;            // [2] the epilogue has read them
    static constexpr int kX = kWEmpty + 2;                // chain 1's (m, l) are there, of an item on both chains
    static constexpr int kDrain = kX + 1;
    static constexpr int kItemFull = kDrain + 1;          // [kPfxItemRing]
    static constexpr int kItemEmpty = kItemFull + kPfxItemRing;
    static constexpr int kNumBars = kItemEmpty + kPfxItemRing;
    static constexpr int kFlagsOff = kBarOff + kNumBars * 8;
    static constexpr int kBytes = kFlagsOff + 16 + kSmemAlign;
    static_assert(kBytes <= kSmemLimit, "shared memory");
    static_assert(2 * kBytes > 233472, "one CTA per SM (each allocates all of TMEM)");
};

// Sequence r: its tokens and keys, and where they begin.  Offsets that do not fit the tensors are clipped.
struct PackedSeq {
    LineSeq line;
    int q0, k0;
};
template <bool PAGED>
__device__ __forceinline__ PackedSeq packed_seq(const PackedParams& p, int r) {
    PackedSeq s;
    s.line.tile_tokens = p.tile_tokens;
    s.line.group = p.G;
    if (PAGED) {
        const int len = __ldg(p.lens + r);
        s.line.nq = len < 0 ? 0 : p.T;
        s.line.nk = min(max(len, 0), p.cap);
        s.line.causal = p.mask == nullptr;
        s.q0 = 0;
        s.k0 = 0;
    } else {
        auto clip = [](int x, int n) { return min(max(x, 0), n); };
        s.q0 = clip(__ldg(p.q_starts + r), p.Nq);
        s.k0 = clip(__ldg(p.k_starts + r), p.Nk);
        s.line.nq = max(0, clip(__ldg(p.q_starts + r + 1), p.Nq) - s.q0);
        s.line.nk = max(0, clip(__ldg(p.k_starts + r + 1), p.Nk) - s.k0);
        s.line.causal = p.causal;
    }
    return s;
}

__device__ __forceinline__ int64_t warp_scan64(int64_t v, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
        const int64_t o = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += o;
    }
    return v;
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ int lds(uint32_t addr) {
    int v;
    asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
// mbar_wait without a call: for the softmax warps, whose registers a call's would not fit beside.  (What they spilled came back
// from L2, since 16 warps' stacks are more than the L1 that the tiles leave: 3000 cycles at each end of an item.)
__device__ __forceinline__ bool mbar_wait_inline(uint32_t bar, uint32_t parity, uint32_t abort_flag, const PackedParams& p) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
#pragma unroll 1
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 31u) == 0) {
            if (lds(abort_flag)) return false;
            if (global_timer_ns() - t0 > p.timeout_ns) {
                atomicCAS(p.error_word, 0u, static_cast<uint32_t>(kDevTimeout));
                asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(abort_flag), "r"(1) : "memory");
                return false;
            }
        }
    }
}

// D (+)= A B with the operands' descriptors given by their low words (start address and leading stride); the
// high word (stride between 8-row groups of 1024 bytes, swizzle) is the same for all of them here.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16); }
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
template <bool ACC>
__device__ __forceinline__ void mma_ss_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "n"(ACC ? 1 : 0), "n"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void mma_ts_lo(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(acc), "n"(kDescHi)
        : "memory");
}

// O_c (+)= P_c V over keys [64 half, 64 half + 64) of a tile of 128; b: V's descriptor.
template <int D>
__device__ __forceinline__ void packed_gemm_full(uint32_t tmem, uint32_t c, uint32_t b, int half, bool first) {
    constexpr uint32_t idesc = make_idesc_bf16_f32(kBr, D, false, true);
    const uint32_t o = tmem + 2 * kBc + c * D, pt = tmem + c * kBc;
#pragma unroll
    for (int kk = half * 4; kk < half * 4 + 4; ++kk)
        mma_ts_lo(o, pt + kk * 8, b + ((kk * 16 * 128) >> 4), idesc, kk > 0 || !first ? 1u : 0u);
}
// ... in steps of 16 of the tile's `steps`.
template <int D>
__device__ __forceinline__ void packed_gemm_o(uint32_t tmem, uint32_t c, uint32_t b, int half, int steps, bool first) {
    constexpr uint32_t idesc = make_idesc_bf16_f32(kBr, D, false, true);
    const uint32_t o = tmem + 2 * kBc + c * D, pt = tmem + c * kBc;
    if (steps == kBc / 16) {
        packed_gemm_full<D>(tmem, c, b, half, first);
    } else {
#pragma unroll 1
        for (int kk = half * 4; kk < min(half * 4 + 4, steps); ++kk)
            mma_ts_lo(o, pt + kk * 8, b + ((kk * 16 * 128) >> 4), idesc, kk > 0 || !first ? 1u : 0u);
    }
}

// One output product with its waits, by the MMA warp.  Not inlined: it has six callers, and the kernel's code is to
// stay within the instruction cache (125 KB of it: every part outside the two loops ran at the
// pace of instruction fetches).  flags: chain, first and last of its item, first and last reader of V, the
// parities of P, O and V.
template <int D>
__device__ __noinline__ bool packed_pv(const WaitCtx& ctx, uint32_t bar0, uint32_t tmem, uint32_t b, uint32_t stage, int steps,
                                       uint32_t flags) {
    using L = PackedSmem<D>;
    auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
    const uint32_t c = flags & 1u;
    bool w = true;
    if (flags & 8u) w = mbar_wait(bar(L::kKvFull + stage), (flags >> 7) & 1u, ctx);
    w = w && mbar_wait(bar(L::kPHalf + c), (flags >> 5) & 1u, ctx);
    if (flags & 2u) w = w && mbar_wait(bar(L::kOEmpty + c), (flags >> 6) & 1u, ctx);
    if (!__all_sync(0xffffffffu, w)) return false;
    tc_fence_after_sync();
    if (elect_one()) packed_gemm_o<D>(tmem, c, b, 0, steps, flags & 2u);
    __syncwarp();
    w = mbar_wait(bar(L::kPFull + c), (flags >> 5) & 1u, ctx);
    if (!__all_sync(0xffffffffu, w)) return false;
    tc_fence_after_sync();
    if (elect_one()) {
        packed_gemm_o<D>(tmem, c, b, 1, steps, flags & 2u);
        if (flags & 16u) mma_commit(bar(L::kKvEmpty + stage));
        if (flags & 4u) mma_commit(bar(L::kOFull + c));
    }
    __syncwarp();
    return true;
}

// Hides the keys of a tile that a row does not see: their scores, in TMEM at t_s, become -infinity, chunk by chunk
// in little code (few tiles need it: the last ones of a unit).  `sees` keys from the tile's first on are seen; or,
// with a row of a mask, those before new token 0, whose key is `-rel` places into the tile, and the new tokens of the row's bits.
static __device__ __noinline__ void packed_hide(uint32_t t_s, int sees, const uint32_t* mask_row, int T, int rel) {
#pragma unroll 1
    for (int i = 0; i < kBc; i += 32) {
        uint32_t seen;  // bit c: key c of the chunk
        if (mask_row != nullptr) {
            const int first = rel + i;  // the chunk's first key among the new tokens
            auto word = [&](int w) -> uint32_t {
                if (w < 0) return 0xffffffffu;  // keys before them
                if (w * 32 >= T) return 0u;
                const uint32_t m = __ldg(mask_row + w);
                return T - w * 32 >= 32 ? m : m & ((1u << (T - w * 32)) - 1u);
            };
            const int w = first >> 5;  // (rounds down)
            seen = __funnelshift_r(word(w), word(w + 1), first & 31);
        } else {
            const int n = sees - i;
            seen = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
        }
        if (__all_sync(0xffffffffu, seen == 0xffffffffu)) continue;
        uint32_t r[32];
        tmem_ld32(t_s + i, r);
        tmem_wait_ld(r);
#pragma unroll
        for (int c = 0; c < 32; ++c)
            if (!(seen & (1u << c))) r[c] = 0xff800000u;  // -infinity
        tmem_st32(t_s + i, r);
    }
    tmem_wait_st();
}

template <int D, bool PAGED>
__global__ void __launch_bounds__(kPkThreads, 1)
attn_packed_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                   const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_kt,
                   const __grid_constant__ CUtensorMap tmap_vt, const __grid_constant__ PackedParams p) {
    using L = PackedSmem<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t s_base = smem_u32(smem);
    const uint32_t bar0 = s_base + L::kBarOff;
    auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kFlagsOff);
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::kFlagsOff + 4);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int lane = threadIdx.x & 31;
    const WaitCtx ctx{abort_flag, p.error_word, p.timeout_ns};
    // For the roles that wait for whole items, whose lengths are the sequences'; they leave with the others before, at an abort.
    const WaitCtx ctx_item{abort_flag, p.error_word, 16 * p.timeout_ns};

    if (threadIdx.x == 0) {
        *abort_flag = 0u;
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(bar(L::kKvFull + s), 1);
            mbar_init(bar(L::kKvEmpty + s), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(L::kQFull + t), 1);
            mbar_init(bar(L::kQEmpty + t), 1);
            mbar_init(bar(L::kSFull + t), 1);
            mbar_init(bar(L::kPHalf + t), 128);
            mbar_init(bar(L::kPFull + t), 128);
            mbar_init(bar(L::kOFull + t), 1);
            mbar_init(bar(L::kOEmpty + t), 128);
            mbar_init(bar(L::kWFull + t), 128);
            mbar_init(bar(L::kWEmpty + t), 128);
        }
        mbar_init(bar(L::kX), 128);
        mbar_init(bar(L::kDrain), 1);
        for (int s = 0; s < kPfxItemRing; ++s) {
            mbar_init(bar(L::kItemFull + s), 1);
            mbar_init(bar(L::kItemEmpty + s), kPkReaders);
        }
        fence_barrier_init();
        tma_prefetch_desc(&tmap_q);
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
        if (!PAGED) {
            tma_prefetch_desc(&tmap_kt);
            tma_prefetch_desc(&tmap_vt);
        }
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    // The combine kernel, where one follows, may be scheduled onto SMs as this grid's CTAs retire;
    // it waits for the whole grid before it reads the partial results.
    if (!p.whole) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // Reads the next item (ring entry n); `it.ntiles` is -1 after the last.  Called by whole warps, whose
    // lanes get one word each from shared memory and hand it round, so that the fields are uniform.
    auto take_item = [&](uint32_t n, PackedItem& it) -> bool {
        const uint32_t s = n % kPfxItemRing;
        if (!__all_sync(0xffffffffu, mbar_wait(bar(L::kItemFull + s), (n / kPfxItemRing) & 1u, ctx))) return false;
        const int* from = reinterpret_cast<const int*>(smem + L::kItemOff + s * sizeof(PackedItem));
        const int word = from[lane < 12 ? lane : 0];
        it.ntiles = __shfl_sync(0xffffffffu, word, 0);
        it.tile0 = __shfl_sync(0xffffffffu, word, 1);
        it.ntiles0 = __shfl_sync(0xffffffffu, word, 2);
        it.klen = __shfl_sync(0xffffffffu, word, 3);
        it.k0 = __shfl_sync(0xffffffffu, word, 4);
        it.req = __shfl_sync(0xffffffffu, word, 5);
        it.head = __shfl_sync(0xffffffffu, word, 6);
        it.tok0 = __shfl_sync(0xffffffffu, word, 7);
        it.nrows = __shfl_sync(0xffffffffu, word, 8);
        it.sees0 = __shfl_sync(0xffffffffu, word, 9);
        it.step = __shfl_sync(0xffffffffu, word, 10);
        it.slot = __shfl_sync(0xffffffffu, word, 11);
        if (lane == 0) mbar_arrive(bar(L::kItemEmpty + s));
        return it.ntiles >= 0;
    };
    // Keys of the item's tile j (1 .. 128).
    auto tile_keys = [](const PackedItem& it, int j) -> int { return min(kBc, it.klen - (it.tile0 + j) * kBc); };

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        RingPos pos{0u, 0u};
        uint32_t issued = 0;
        bool ok = true;
        PackedItem it;
#pragma unroll 1
        for (uint32_t n = 0; ok && take_item(n, it); ++n) {
            const int* pages = PAGED ? p.table + it.req * p.table_stride : nullptr;
            // paged: lane l holds the page of box `base + l` of the item's keys, and has asked for the next 32
            const int box0 = PAGED ? it.tile0 * (kBc / p.box) : 0;
            const int boxes_all = PAGED ? (it.klen + p.box - 1) / p.box : 0;
            auto page_of = [&](int bx) -> int {
                const int key = bx * p.box;
                const int page = bx < boxes_all ? __ldg(pages + (key >> p.page_log2)) : 0;
                return static_cast<uint32_t>(page) < static_cast<uint32_t>(p.pages) ? page : p.pages;
            };
            int base = box0, page_now = 0, page_next = 0;
            if (PAGED && it.ntiles > 0) {
                page_now = page_of(base + lane);
                page_next = page_of(base + 32 + lane);
            }
#pragma unroll 1
            for (int j = 0; j < it.ntiles && ok; ++j) {
                const int keys = tile_keys(it, j);
                const int key = (it.tile0 + j) * kBc;
                int my_page = 0, nbox = 0;
                if (PAGED) {
                    // boxes of a tile are at most 8, so a run of 32 holds whole tiles
                    const int b = key / p.box;
                    if (b >= base + 32) {
                        base += 32;
                        page_now = page_next;
                        page_next = page_of(base + 32 + lane);
                    }
                    nbox = (keys + p.box - 1) / p.box;
                    my_page = __shfl_sync(0xffffffffu, page_now, (b - base + lane) & 31);
                }
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kKvEmpty + pos.stage), pos.phase ^ 1u, ctx));
                    if (!ok) break;
                    const uint32_t full = bar(L::kKvFull + pos.stage);
                    const uint32_t dst = s_base + L::kRingOff + pos.stage * L::kTile;
                    if (PAGED) {
                        if (lane == 0) mbar_arrive_expect_tx(full, nbox * p.box * D * 2);
                        __syncwarp();
                        if (lane < nbox) {  // page p.pages: outside the cache, reads as zero
                            const int within = (key + lane * p.box) & ((1 << p.page_log2) - 1);
#pragma unroll
                            for (int b = 0; b < D / 64; ++b)
                                tma_load_4d(dst + b * (kBc * 128) + lane * p.box * 128, kv == 0 ? &tmap_k : &tmap_v, full,
                                            b * 64, within, it.head, my_page);
                        }
                        __syncwarp();
                    } else if (elect_one()) {
                        if (keys == kBc) {
                            mbar_arrive_expect_tx(full, L::kTile);
#pragma unroll
                            for (int b = 0; b < D / 64; ++b)
                                tma_load_3d(dst + b * (kBc * 128), kv == 0 ? &tmap_k : &tmap_v, full, b * 64, it.k0 + key,
                                            it.head);
                        } else {
                            const int boxes = (keys + kPkTailBox - 1) / kPkTailBox;
                            mbar_arrive_expect_tx(full, boxes * kPkTailBox * D * 2);
#pragma unroll 1
                            for (int i = 0; i < boxes; ++i)
#pragma unroll
                                for (int b = 0; b < D / 64; ++b)
                                    tma_load_3d(dst + b * (kBc * 128) + i * (kPkTailBox * 128), kv == 0 ? &tmap_kt : &tmap_vt,
                                                full, b * 64, it.k0 + key + i * kPkTailBox, it.head);
                        }
                    }
                    __syncwarp();
                    pos = pos.next(L::kStages);
                    ++issued;
                }
            }
        }
        // every issued copy lands before the CTA's shared memory is released (bounded waits)
        const uint32_t pending = issued < static_cast<uint32_t>(L::kStages) ? issued : L::kStages;
        RingPos back = pos;
#pragma unroll 1
        for (uint32_t i = 0; i < pending; ++i) {
            back = back.stage == 0 ? RingPos{L::kStages - 1u, back.phase ^ 1u} : RingPos{back.stage - 1, back.phase};
            mbar_wait_drain(bar(L::kKvFull + back.stage), back.phase, 50000000ull);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        const uint32_t idesc_s = make_idesc_bf16_f32(kBr, kBc, false, false) | (p.negate_scores ? kIdescNegateB : 0u);
        constexpr uint32_t kTile16 = L::kTile >> 4;
        const uint32_t dq0 = desc_lo(s_base + L::kQOff, 16);
        const uint32_t dk0 = desc_lo(s_base + L::kRingOff, 16);
        const uint32_t dv0 = desc_lo(s_base + L::kRingOff, kBc * 128);
        uint32_t p_phase = 0u, o_phase = 3u;  // parities to wait for, bit c of chain c
        RingPos kpos{0u, 0u};   // K of the current tile
        uint32_t qpos = 0;      // query tiles taken so far: slot qpos & 1
        uint32_t par = 0;       // chain of the item's first step
        bool ok = true;
        // S_c = Q K^T
        auto gemm_s = [&](int c, uint32_t a, uint32_t b) {
            mma_ss_lo<false>(tmem + c * kBc, a, b, idesc_s);
#pragma unroll
            for (int kk = 1; kk < D / 16; ++kk) {
                const uint32_t off = static_cast<uint32_t>(((kk >> 2) * (kBr * 128) + (kk & 3) * 32) >> 4);
                mma_ss_lo<true>(tmem + c * kBc, a + off, b + off, idesc_s);
            }
        };
        // the output product that is due: of the step before
        struct { bool due, first, last, first_v, last_v; int chain, ksteps; RingPos v; } pv{};
        auto run_pv = [&]() -> bool {
            if (!pv.due) return true;
            pv.due = false;
            const uint32_t c = pv.chain;
            const uint32_t flags = c | (pv.first ? 2u : 0u) | (pv.last ? 4u : 0u) | (pv.first_v ? 8u : 0u) | (pv.last_v ? 16u : 0u) |
                                   (((p_phase >> c) & 1u) << 5) | (((o_phase >> c) & 1u) << 6) | (pv.v.phase << 7);
            p_phase ^= 1u << c;
            if (pv.first) o_phase ^= 1u << c;
            return packed_pv<D>(ctx, bar0, tmem, dv0 + pv.v.stage * kTile16, pv.v.stage, pv.ksteps, flags);
        };
        // The next score product goes first where its operands are there already: the tensor core
        // works on it while the softmax of the step before runs.  Where they are not (short items,
        // the ends of a CTA's share), the product that is due does not wait for them.
        auto there = [&](uint32_t b, uint32_t parity) -> bool { return __all_sync(0xffffffffu, mbar_test(b, parity)); };
        PackedItem it;
#pragma unroll 1
        for (uint32_t n = 0; ok; ++n) {
            if (pv.due && !there(bar(L::kItemFull + n % kPfxItemRing), (n / kPfxItemRing) & 1u) && !(ok = run_pv())) break;
            if (!take_item(n, it)) break;
            const int nt = it.ntiles;
            if (nt == 0) continue;
            if (it.nrows > p.qrows) {
                // Two query tiles, chain = tile: S0_j; O1 += P1_{j-1} V_{j-1}; S1_j; O0 += P0_j V_j, the
                // first of them over the first n0 K/V tiles (causal: it may see one tile less).
                const int n0 = it.ntiles0;
                const uint32_t q0 = qpos & 1u, q1 = q0 ^ 1u;
                if (pv.due && (pv.chain == 0 || !there(bar(L::kKvFull + kpos.stage), kpos.phase) ||
                               !there(bar(L::kQFull + q0), (qpos >> 1) & 1u)) && !(ok = run_pv()))
                    break;
                const uint32_t a0 = dq0 + q0 * kTile16, a1 = dq0 + q1 * kTile16;
                const int last_steps = (tile_keys(it, nt - 1) + 15) / 16;
                // O_c (+)= P_c V_j for a tile of 128 keys, V_j at ring position v.  Inlined, without a tail's conditions:
                // this warp's own instructions bound the loop (with the products behind a call, 2175 -> 2494 us on long documents).
                auto pv_full = [&](auto chain, bool first, RingPos v) -> bool {
                    constexpr int c = decltype(chain)::value;
                    bool w = true;
                    if (c == 0) w = mbar_wait(bar(L::kKvFull + v.stage), v.phase, ctx);  // (chain 1 follows)
                    w = w && mbar_wait(bar(L::kPHalf + c), (p_phase >> c) & 1u, ctx);
                    if (first) {
                        w = w && mbar_wait(bar(L::kOEmpty + c), (o_phase >> c) & 1u, ctx);
                        o_phase ^= 1u << c;
                    }
                    if (!__all_sync(0xffffffffu, w)) return false;
                    tc_fence_after_sync();
                    const uint32_t b = dv0 + v.stage * kTile16;
                    if (elect_one()) packed_gemm_full<D>(tmem, c, b, 0, first);
                    __syncwarp();
                    w = mbar_wait(bar(L::kPFull + c), (p_phase >> c) & 1u, ctx);
                    p_phase ^= 1u << c;
                    if (!__all_sync(0xffffffffu, w)) return false;
                    tc_fence_after_sync();
                    if (elect_one()) {
                        packed_gemm_full<D>(tmem, c, b, 1, false);
                        if (c == 1) mma_commit(bar(L::kKvEmpty + v.stage));
                    }
                    __syncwarp();
                    return true;
                };
                RingPos vprev{0u, 0u};
#pragma unroll 1
                for (int j = 0; j < nt && ok; ++j) {
                    bool w = mbar_wait(bar(L::kKvFull + kpos.stage), kpos.phase, ctx);
                    if (j == 0)
                        w = w && mbar_wait(bar(L::kQFull + q0), (qpos >> 1) & 1u, ctx) &&
                            mbar_wait(bar(L::kQFull + q1), ((qpos + 1) >> 1) & 1u, ctx);
                    if (!(ok = __all_sync(0xffffffffu, w))) break;
                    const uint32_t b = dk0 + kpos.stage * kTile16;
                    if (j < n0) {
                        if (elect_one()) {
                            gemm_s(0, a0, b);
                            mma_commit(bar(L::kSFull + 0));
                            if (j == n0 - 1) mma_commit(bar(L::kQEmpty + q0));
                        }
                        __syncwarp();
                    }
                    // (chain 0 took every tile before the last, so that V_{j-1} is there, and only the last may have a tail;
                    // where chain 0 ends before it, its O is complete here)
                    ok = j == 0 ? run_pv() : pv_full(std::integral_constant<int, 1>{}, j == 1, vprev);
                    if (!ok) break;
                    if (elect_one()) {
                        gemm_s(1, a1, b);
                        mma_commit(bar(L::kSFull + 1));
                        mma_commit(bar(L::kKvEmpty + kpos.stage));
                        if (j == nt - 1) mma_commit(bar(L::kQEmpty + q1));
                        if (j == n0) mma_commit(bar(L::kOFull + 0));
                    }
                    __syncwarp();
                    vprev = kpos.next(L::kStages);
                    if (j < nt - 1) {
                        if (!(ok = pv_full(std::integral_constant<int, 0>{}, j == 0, vprev))) break;
                    } else if (n0 == nt) {
                        pv.due = true;
                        pv.chain = 0;
                        pv.v = vprev;
                        pv.ksteps = last_steps;
                        pv.first = nt == 1;
                        pv.last = true;
                        pv.first_v = true;
                        pv.last_v = false;
                        if (!(ok = run_pv())) break;
                    }
                    kpos = vprev.next(L::kStages);
                }
                if (!ok) break;
                pv.due = true;
                pv.chain = 1;
                pv.v = vprev;
                pv.ksteps = last_steps;
                pv.first = nt == 1;
                pv.last = true;
                pv.first_v = nt > n0;
                pv.last_v = true;
                qpos += 2;
                par = 0;
                continue;
            }
            // One query tile; the chains take turns with the K/V tiles.
            const uint32_t qslot = qpos & 1u;
#pragma unroll 1
            for (int j = 0; j < nt && ok; ++j) {
                const int c = (par + j) & 1;
                if (pv.due && (!there(bar(L::kKvFull + kpos.stage), kpos.phase) ||
                               (j == 0 && !there(bar(L::kQFull + qslot), (qpos >> 1) & 1u))) && !(ok = run_pv()))
                    break;
                bool w = mbar_wait(bar(L::kKvFull + kpos.stage), kpos.phase, ctx);
                if (j == 0) w = w && mbar_wait(bar(L::kQFull + qslot), (qpos >> 1) & 1u, ctx);
                if (!(ok = __all_sync(0xffffffffu, w))) break;
                if (elect_one()) {
                    gemm_s(c, dq0 + qslot * kTile16, dk0 + kpos.stage * kTile16);
                    mma_commit(bar(L::kSFull + c));
                    mma_commit(bar(L::kKvEmpty + kpos.stage));
                    if (j == nt - 1) mma_commit(bar(L::kQEmpty + qslot));
                }
                __syncwarp();
                if (!(ok = run_pv())) break;
                pv.due = true;
                pv.chain = c;
                pv.v = kpos.next(L::kStages);
                pv.ksteps = (tile_keys(it, j) + 15) / 16;
                pv.first = j < 2;
                pv.last = j + 2 >= nt;
                pv.first_v = true;
                pv.last_v = true;
                kpos = pv.v.next(L::kStages);
            }
            ++qpos;
            par = (par + nt) & 1u;
        }
        if (ok) run_pv();
        // Make sure no MMA is still writing TMEM when it is released.
        if (elect_one()) mma_commit(bar(L::kDrain));
        __syncwarp();
        mbar_wait_drain(bar(L::kDrain), 0, 1000000000ull);
    } else if (warp == 2) {
        // ------------------------------------------------------------ scheduler
        uint32_t n = 0;
        bool ok = true;
        auto publish = [&](const PackedItem& it) {
            const uint32_t s = n % kPfxItemRing;
            if (n >= kPfxItemRing) ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kItemEmpty + s), ((n / kPfxItemRing) - 1) & 1u, ctx_item));
            if (!ok) return;
            if (lane == 0) {
                *reinterpret_cast<PackedItem*>(smem + L::kItemOff + s * sizeof(PackedItem)) = it;
                mbar_arrive(bar(L::kItemFull + s));
            }
            __syncwarp();
            ++n;
        };
        PackedItem it{};
        // The line's length: each lane sums a run of sequences (up to 32 of them: has one, and keeps it).
        const int run = (p.R + 31) / 32;
        int64_t mine = 0;
        PackedSeq own{};
        int64_t own_len = 0;
        int most_keys = 0, most_tokens = 0;
#pragma unroll 1
        for (int i = 0; i < run; ++i) {
            const int r = lane * run + i;
            if (r < p.R) {
                own = packed_seq<PAGED>(p, r);
                own_len = own.line.length();
                mine += own_len;
                if (own.line.nq > 0) most_keys = max(most_keys, own.line.nk);
                most_tokens = max(most_tokens, min(own.line.nq, own.line.block_tokens()));
            }
        }
        mine *= p.Hk;
        const int64_t upto = warp_scan64(mine, lane);
        const int64_t total = __shfl_sync(0xffffffffu, upto, 31);
        const int64_t len = line_stretch(total, p.stretches);
        const bool whole = p.whole || line_whole(__reduce_max_sync(0xffffffffu, most_keys),
                                                  __reduce_max_sync(0xffffffffu, most_tokens) * p.G, len);
        // (after a timeout too: what the merging kernel reads of the cuts has to be theirs)
#pragma unroll 1
        for (int i = blockIdx.x; i < p.stretches; i += gridDim.x) {
            const int64_t x0 = i * len;
            const int64_t x1 = min(x0 + len, total);
            PackedCut cut{};
            if (ok && x0 < x1) {
                // the run of sequences that x0 is in, then the sequences in groups of 32
                const int at = run == 1 ? 0 : __ffs(__ballot_sync(0xffffffffu, upto > x0)) - 1;
                int64_t start = __shfl_sync(0xffffffffu, upto - mine, at);
#pragma unroll 1
                for (int r0 = at * run; r0 < p.R && start < x1 && ok; r0 += 32) {
                    if (run > 1) {
                        own_len = 0;
                        if (r0 + lane < p.R) {
                            own = packed_seq<PAGED>(p, r0 + lane);
                            own_len = own.line.length();
                        }
                    }
                    const int64_t cost = own_len * p.Hk;
                    const int64_t end_l = start + warp_scan64(cost, lane);
                    uint32_t in = __ballot_sync(0xffffffffu, cost > 0 && end_l > x0 && end_l - cost < x1);
#pragma unroll 1
                    for (; in != 0 && ok; in &= in - 1) {
                        const int src = __ffs(in) - 1;
                        PackedSeq s;
                        s.line.nq = __shfl_sync(0xffffffffu, own.line.nq, src);
                        s.line.nk = __shfl_sync(0xffffffffu, own.line.nk, src);
                        s.line.tile_tokens = p.tile_tokens;
                        s.line.group = p.G;
                        s.line.causal = PAGED ? p.mask == nullptr : p.causal;
                        s.q0 = __shfl_sync(0xffffffffu, own.q0, src);
                        s.k0 = __shfl_sync(0xffffffffu, own.k0, src);
                        const int64_t first = __shfl_sync(0xffffffffu, end_l - cost, src);
                        const int64_t per = __shfl_sync(0xffffffffu, own_len, src);
                        const int nb = s.line.blocks();
                        it.req = r0 + src;
                        it.k0 = s.k0;
                        it.step = s.line.causal ? 1 : 0;
                        int h = x0 > first ? static_cast<int>(line_div(x0 - first, per)) : 0;
#pragma unroll 1
                        for (int64_t hs = first + h * per; h < p.Hk && hs < x1 && ok; ++h, hs += per) {
                            // the block that x0 is in: the last one that begins at or before it
                            int b = 0;
                            if (x0 > hs) {
                                int lo = 0, hi = nb;  // before(lo) <= x0 - hs, and not before(hi)
                                while (hi - lo > 1) {
                                    const int width = (hi - lo + 31) / 32;
                                    const int probe = lo + lane * width;
                                    const bool below = probe < hi && s.line.before(probe) <= x0 - hs;
                                    const int k = 31 - __clz(__ballot_sync(0xffffffffu, below));  // lane 0 is
                                    lo += k * width;
                                    hi = min(hi, lo + width);
                                }
                                b = lo;
                            }
                            int64_t us = hs + s.line.before(b);
#pragma unroll 1
                            for (; b < nb && us < x1 && ok; ++b) {
                                const int tok0 = b * s.line.block_tokens(), tokens = s.line.tokens(b);
                                const int klen = s.line.keys(b);
                                const int tiles = (klen + kBc - 1) / kBc;
                                const int64_t begin = us + s.line.unit_cost(b);
                                LinePart part(begin, tiles, kLineTile, x0, x1);
                                // A whole unit is the stretch's that its middle is in, so that equal units come one to a stretch (by
                                // their beginnings 1200 tokens at 32 heads of 8, full attention, took 42 us, 27 like this).
                                const int64_t mark = whole ? us + (s.line.unit_cost(b) + klen) / 2 : us;
                                const bool mine_all = mark >= x0 && mark < x1;
                                if (whole) {
                                    part.t0 = mine_all ? 0 : tiles;
                                    part.t1 = tiles;
                                }
                                const bool none = tiles == 0 && mine_all;  // nothing seen: only written
                                if (part.t0 < part.t1 || none) {
                                    it.ntiles = tiles == 0 ? 0 : part.t1 - part.t0;
                                    it.tile0 = tiles == 0 ? 0 : part.t0;
                                    it.klen = klen;
                                    it.head = h;
                                    it.tok0 = s.q0 + tok0;
                                    it.nrows = tokens * p.G;
                                    it.sees0 = it.step ? tok0 - s.line.nq + s.line.nk + 1 : klen;  // (in this order: in 32 bits)
                                    it.ntiles0 = it.ntiles;
                                    if (tokens > s.line.tile_tokens && it.ntiles > 0) {  // at least one, which it may not see a key of
                                        const int seen0 = s.line.sees(tok0 + s.line.tile_tokens - 1);
                                        it.ntiles0 = max(1, min(it.ntiles, (seen0 + kBc - 1) / kBc - it.tile0));
                                    }
                                    it.slot = -1;
                                    if (tiles > 0 && it.ntiles < tiles) {
                                        it.slot = it.tile0 == 0 ? 2 * i + 1 : 2 * i;
                                        if (it.tile0 == 0) {
                                            const int64_t last = begin + static_cast<int64_t>(tiles - 1) * kLineTile;
                                            cut.pieces = static_cast<int>(line_div(last, len)) - i + 1;
                                            cut.head = h;
                                            cut.req = it.req;
                                            cut.tok0 = it.tok0;
                                            cut.nrows = it.nrows;
                                        }
                                    }
                                    publish(it);
                                }
                                us += s.line.cost(b);
                            }
                        }
                    }
                    start = __shfl_sync(0xffffffffu, end_l, 31);
                }
            }
            if (lane == 0 && !p.whole) p.cuts[i] = cut;
        }
        it.ntiles = -1;
        if (ok) publish(it);
    } else if (warp == 3) {
        // ------------------------------------------------------------ Q loader
        uint32_t qpos = 0;
        uint32_t q_slots = 0, q_parity = 0;  // slots that a copy was issued to, and the parity it completes
        bool ok = true;
        PackedItem it;
#pragma unroll 1
        for (uint32_t n = 0; ok && take_item(n, it); ++n) {
            if (it.ntiles == 0) continue;
#pragma unroll 1
            for (int k = 0; k < (it.nrows > p.qrows ? 2 : 1) && ok; ++k, ++qpos) {
                const uint32_t slot = qpos & 1u;
                ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kQEmpty + slot), ((qpos >> 1) & 1u) ^ 1u, ctx_item));
                if (!ok) break;
                const uint32_t full = bar(L::kQFull + slot);
                if (lane == 0) {  // whole tokens; what lies behind the tensor reads as zero
                    mbar_arrive_expect_tx(full, p.qrows * D * 2);
                    if (!(p.withhold_first_q && blockIdx.x % 2 == 0 && qpos == 0)) {
#pragma unroll
                        for (int b = 0; b < D / 64; ++b)
                            tma_load_5d(s_base + L::kQOff + slot * L::kTile + b * (kBr * 128), &tmap_q, full, b * 64, 0, it.head,
                                        it.tok0 + k * p.tile_tokens, PAGED ? it.req : 0);
                    }
                }
                q_slots |= 1u << slot;
                q_parity = (q_parity & ~(1u << slot)) | (((qpos >> 1) & 1u) << slot);
                __syncwarp();
            }
        }
#pragma unroll 1
        for (uint32_t s = 0; s < 2; ++s)  // the copies land before the shared memory is released
            if (q_slots & (1u << s)) mbar_wait_drain(bar(L::kQFull + s), (q_parity >> s) & 1u, 50000000ull);
    } else if (warp < 12) {
        // ------------------------------------------------------------ softmax warpgroups
        auto inline_wait = [&](uint32_t b, uint32_t parity) { return mbar_wait_inline(b, parity, s_base + L::kFlagsOff + 4, p); };
        const int t = (warp - 4) >> 2;          // chain
        const int quad = warp & 3;              // TMEM lane quadrant
        const int rloc = quad * 32 + lane;      // row within the tile
        const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t t_s = tmem + lane_addr + t * kBc;
        const uint32_t t_o = tmem + lane_addr + 2 * kBc;  // O_0; O_1 is D columns further
        const float sl2 = p.scale_log2;
        uint32_t ring = 0;   // K/V fills before this item
        // Bits: parity of the next S; of the next item on both chains; of chain c's next item; the chain of the next item's first step.
        constexpr uint32_t kS = 1, kXBit = 1, kOBit = 2, kParBit = 4;
        uint32_t state = 0;
        bool ok = true;
        // An item's fields stay in its ring entry, to be read where they are needed (and again at its end): held in
        // registers beside the scores they were spilled, and 16 warps' stacks are more than the L1 that the tiles leave.
#pragma unroll 1
        for (uint32_t n = 0; ok; ++n) {
            const uint32_t entry = n % kPfxItemRing;
            auto field = [&](size_t at) -> int {
                return lds(s_base + L::kItemOff + entry * static_cast<uint32_t>(sizeof(PackedItem)) + static_cast<uint32_t>(at));
            };
            if (!__all_sync(0xffffffffu, inline_wait(bar(L::kItemFull + entry), (n / kPfxItemRing) & 1u))) break;
            const int nt = field(offsetof(PackedItem, ntiles));
            if (nt < 0) break;
            const bool two = field(offsetof(PackedItem, nrows)) > p.qrows;
            const bool both = two || nt >= 2;                 // both chains work on the item
            // an item of one query tile: this chain's first K/V tile (two query tiles: chain t has tile t)
            const int mine = two ? 0 : t ^ static_cast<int>((state >> kParBit) & 1u);
            float m_ref = -INFINITY;
            float l = 0.f;
            if (nt > 0 && (both || mine == 0)) {
                const int nt_mine = two && t == 0 ? field(offsetof(PackedItem, ntiles0)) : nt;
                const int nrow = min(p.qrows, field(offsetof(PackedItem, nrows)) - (two ? t * p.qrows : 0));
                const bool warp_on = quad * 32 < nrow;            // the warp has rows
                const bool row_on = rloc < nrow;
                // Key counts from the item's first tile on: all that the unit sees, those that this row
                // sees and that every row of the tile does.
                const int left = field(offsetof(PackedItem, klen)) - field(offsetof(PackedItem, tile0)) * kBc;
                int lim, all_see;
                const uint32_t* mask_row = nullptr;
                if (PAGED && p.mask) {
                    lim = left;
                    all_see = left - p.T;  // where the new tokens' keys begin
                    const int tok = field(offsetof(PackedItem, tok0)) + (two ? t * p.tile_tokens : 0) + (row_on ? rloc / p.G : 0);
                    mask_row = p.mask + (static_cast<int64_t>(field(offsetof(PackedItem, req))) * p.T + tok) * p.words;
                } else {
                    const int tile_tok = two ? t * p.tile_tokens : 0;
                    const int sees = field(offsetof(PackedItem, sees0)) - field(offsetof(PackedItem, tile0)) * kBc, step = field(offsetof(PackedItem, step));
                    lim = min(left, sees + (tile_tok + rloc / p.G) * step);
                    all_see = min(left, sees + tile_tok * step);
                }
                bool first = true;
#pragma unroll 1
                for (int j = mine; j < nt_mine; j += two ? 1 : 2) {
                    ok = __all_sync(0xffffffffu, inline_wait(bar(L::kSFull + t), state & kS));
                    state ^= kS;
                    if (!ok) break;
                    tc_fence_after_sync();
                    const int key0 = j * kBc;
                    const int keys = min(kBc, left - key0);
                    // The output product sums over keys in steps of 16.  What lies behind the last key may
                    // hold anything (a NaN times a zero weight is a NaN): zero it, before the first product that reads it.
                    if ((keys & 15) != 0 && (!two || t == (j < field(offsetof(PackedItem, ntiles0)) ? 0 : 1))) {
                        const uint32_t at = ring + 2 * j + 1;  // V_j's fill
                        const uint32_t stage = at % L::kStages;
                        ok = __all_sync(0xffffffffu, inline_wait(bar(L::kKvFull + stage), (at / L::kStages) & 1u));
                        if (!ok) break;
                        const int pad = ((keys + 15) & ~15) - keys;
                        const uint32_t v = s_base + L::kRingOff + stage * L::kTile;
#pragma unroll 1
                        for (int i = rloc; i < pad * (D / 8); i += 128) {
                            const int row = keys + i / (D / 8), c8 = i % (D / 8);
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(v + (c8 >> 3) * (kBc * 128) + row * 128 + (c8 & 7) * 16), "r"(0) : "memory");
                        }
                        fence_proxy_async_smem();
                    }
                    if (!warp_on) {  // none of this warp's rows exist: only keep the barriers' counts
                        mbar_arrive(bar(L::kPHalf + t));
                        mbar_arrive(bar(L::kPFull + t));
                        continue;
                    }
                    const float m_old = m_ref;
                    bool grow = false;
                    float alpha = 1.f;
                    // moves the reference maximum and l where a tile's maximum asks for it
                    auto refer = [&](float mx) {
                        // a row that sees no key of the tile keeps its reference (0 * -inf would be a NaN)
                        const float m_tile = mx == -INFINITY ? -INFINITY : mx * p.max_scale_log2;
                        grow = row_on && m_tile > m_old + kRescaleLog2Bf16;
                        if (grow) {
                            alpha = ex2_approx(m_old - m_tile);  // 0 the first time
                            m_ref = m_tile;
                        }
                        l *= alpha;
                    };
                    // Rescales O when a reference moved, before the first half of P is released.
                    // O's previous product has completed: it was issued before this S.
                    auto rescale = [&]() {
                        if (__any_sync(0xffffffffu, grow && !first)) {
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                uint32_t o[32];
                                tmem_ld32(t_o + t * D + c, o);
                                tmem_wait_ld(o);
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                                tmem_st32(t_o + t * D + c, o);
                            }
                        }
                        first = false;
                    };
                    float acc0 = 0.f, acc1 = 0.f, acc2 = 0.f, acc3 = 0.f;
                    // P = 2^(s scale log2 e - m) of 16 keys, as bf16 pairs over the scores' first half
                    auto exp_chunk = [&](const uint32_t (&r)[16], uint32_t col) {
                        const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
                        uint32_t pk[8];
#pragma unroll
                        for (int c = 0; c < 8; c += 2) {
                            float x0, x1, x2, x3;
                            ffma2(x0, x1, __uint_as_float(r[2 * c]), __uint_as_float(r[2 * c + 1]), sl2, -m_use);
                            ffma2(x2, x3, __uint_as_float(r[2 * c + 2]), __uint_as_float(r[2 * c + 3]), sl2, -m_use);
                            const float a0 = ex2_approx(x0), b0 = ex2_approx(x1);
                            const float a1 = ex2_approx(x2), b1 = ex2_approx(x3);
                            fadd2(acc0, acc1, a0, b0);
                            fadd2(acc2, acc3, a1, b1);
                            pk[c] = pack_bf16x2(a0, b0);
                            pk[c + 1] = pack_bf16x2(a1, b1);
                        }
                        tmem_st8(t_s + col, pk);
                    };
                    const bool masked = key0 + kBc > all_see;  // some row does not see all 128 keys
                    if (masked) packed_hide(t_s, lim - key0, PAGED && p.mask ? mask_row : nullptr, p.T, key0 - all_see);
                    // With 16 warps a thread has 128 registers, half of what the scores and their exponentials would
                    // take: they are read for the maximum, and again 16 keys ahead of the exponentials (32 ahead, a thread
                    // spilled 20 registers more: 24 prompts of 20 to 2000 tokens in 250 us, 234 like this).
                    uint32_t ra[32], rb[32];
                    auto largest = [](const uint32_t (&r)[32]) {
                        const float* sc = reinterpret_cast<const float*>(r);
                        float m0 = fmax3(sc[0], sc[1], sc[2]), m1 = fmax3(sc[3], sc[4], sc[5]);
#pragma unroll
                        for (int c = 6; c < 30; c += 4) {
                            m0 = fmax3(m0, sc[c], sc[c + 1]);
                            m1 = fmax3(m1, sc[c + 2], sc[c + 3]);
                        }
                        return fmax3(m0, m1, fmaxf(sc[30], sc[31]));
                    };
                    tmem_ld32(t_s + 64, ra);
                    tmem_ld32(t_s + 96, rb);
                    tmem_wait_ld(ra);
                    tmem_wait_ld(rb);
                    float mx = largest(ra);
                    tmem_ld32(t_s + 0, ra);
                    mx = fmaxf(mx, largest(rb));
                    tmem_ld32(t_s + 32, rb);
                    tmem_wait_ld(ra);
                    tmem_wait_ld(rb);
                    refer(fmax3(mx, largest(ra), largest(rb)));
                    rescale();
                    auto half_done = [&]() {  // keys 0-63
                        tmem_wait_st();
                        tc_fence_before_sync();
                        mbar_arrive(bar(L::kPHalf + t));
                    };
                    {
                        uint32_t s0[16], s1[16];
                        tmem_ld16(t_s, s0);
                        tmem_wait_ld16(s0);
#pragma unroll
                        for (int i = 0; i < 8; i += 2) {
                            tmem_ld16(t_s + 16 * (i + 1), s1);
                            exp_chunk(s0, 8 * i);
                            tmem_wait_ld16(s1);
                            if (i + 2 < 8) tmem_ld16(t_s + 16 * (i + 2), s0);
                            exp_chunk(s1, 8 * (i + 1));
                            if (i == 2) half_done();
                            if (i + 2 < 8) tmem_wait_ld16(s0);
                        }
                    }
                    l += (acc0 + acc1) + (acc2 + acc3);
                    tmem_wait_st();
                    tc_fence_before_sync();
                    mbar_arrive(bar(L::kPFull + t));
                }
                if (!ok) break;
                // The rows' weights for the epilogue, 1 / l, and the log-sum-exp.
                const bool merge = both && !two;
                float* weight = reinterpret_cast<float*>(smem + L::kWeightOff) + rloc;
                float2* pair = reinterpret_cast<float2*>(smem + L::kWeightOff) + rloc;
                float w_own = 1.f, w_other = 0.f;  // of this chain's O and the other's
                float m = m_ref, sum = l;
                ok = inline_wait(bar(L::kWEmpty + t), ((state >> (kOBit + t)) & 1u) ^ 1u);
                if (merge) {
                    if (t == 1) {  // its (m, l) lie where the other tile's weights would
                        ok = ok && inline_wait(bar(L::kWEmpty + 0), ((state >> kOBit) & 1u) ^ 1u);
                        if (ok) *pair = make_float2(m_ref, l);
                        mbar_arrive(bar(L::kX));
                    } else {
                        // (a barrier of its own, counted by such items: chain 0 may be items ahead of chain 1)
                        ok = ok && inline_wait(bar(L::kX), (state >> kXBit) & 1u);
                        const float2 other = *pair;
                        m = fmaxf(m_ref, other.x);
                        w_own = m_ref == -INFINITY ? 0.f : ex2_approx(m_ref - m);
                        w_other = other.x == -INFINITY ? 0.f : ex2_approx(other.x - m);
                        // a chain whose reference never moved has l = 0, or a NaN to pass on
                        sum = (m_ref == -INFINITY ? l : l * w_own) + (other.x == -INFINITY ? other.y : other.y * w_other);
                    }
                    state ^= 1u << kXBit;
                }
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                if (!merge || t == 0) {
                    // A row that sees no key of this piece: LSE = -inf, and a weight of -0 says that O is 0
                    // (0 times a NaN of V would not be).
                    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? -0.f : sum);
                    if (merge) *pair = sum == 0.f ? make_float2(-0.f, 0.f) : make_float2(w_own * inv, w_other * inv);
                    else weight[t * 128] = inv;
                }
                mbar_arrive(bar(L::kWFull + t));
                if (row_on && (!merge || t == 0)) {
                    const float lse = sum == 0.f ? -INFINITY : (m + lg2_approx(sum)) * kLn2;
                    const int slot = field(offsetof(PackedItem, slot));
                    float* to;
                    if (slot < 0) {
                        const int row_tok = rloc / p.G;
                        const int tok = field(offsetof(PackedItem, tok0)) + (two ? t * p.tile_tokens : 0) + row_tok, hq = field(offsetof(PackedItem, head)) * p.G + rloc - row_tok * p.G;
                        to = p.lse + (PAGED ? field(offsetof(PackedItem, req)) * p.ls[0] : 0) + hq * p.ls[1] + tok;
                    } else {
                        to = p.part_lse + static_cast<int64_t>(slot) * p.orows + (two ? t * p.qrows : 0) + rloc;
                    }
                    *to = lse;
                }
            }
            __syncwarp();  // every lane has read the ring entry
            if (lane == 0) mbar_arrive(bar(L::kItemEmpty + entry));
            if (nt == 0) continue;
            const uint32_t par = (state >> kParBit) & 1u;
            state ^= (both ? 3u : 1u << par) << kOBit;
            ring += 2 * nt;
            state = (state & ~(1u << kParBit)) | ((two ? 0u : (par + nt) & 1u) << kParBit);
        }
    } else {
        // ------------------------------------------------------------ epilogue
        // Thread r of the warpgroup has row r of a tile.  (Exchanges among threads that would make the stores of a row
        // neighbours cost more than the stores: 9400 cycles for a unit's two tiles, 4500 like this, at d = 128.)
        const int quad = warp & 3;
        const int rloc = quad * 32 + lane;
        const uint32_t t_o = tmem + (static_cast<uint32_t>(quad * 32) << 16) + 2 * kBc;
        const float* weight = reinterpret_cast<const float*>(smem + L::kWeightOff);
        const int row_tok = rloc / p.G, row_head = rloc - row_tok * p.G;
        uint32_t o_phase = 0u, par = 0;
        bool ok = true;
        PackedItem it;
#pragma unroll 1
        for (uint32_t n = 0; ok && take_item(n, it); ++n) {
            const bool two = it.nrows > p.qrows;
            const int nt = it.ntiles;
            const bool merge = !two && nt >= 2;
#pragma unroll 1
            for (int k = 0; k < (two ? 2 : 1) && ok; ++k) {
                const int c = two ? k : merge ? 0 : static_cast<int>(par);  // chain
                const int nrow = min(p.qrows, it.nrows - k * p.qrows);
                const bool row_on = rloc < nrow;
                const int tok = it.tok0 + k * p.tile_tokens + row_tok, hq = it.head * p.G + row_head;
                const int64_t req = PAGED ? it.req : 0;
                uint4* out = reinterpret_cast<uint4*>(p.o + req * p.os[0] + hq * p.os[1] + tok * p.os[2]);
                if (nt == 0) {  // no key for any row: O = 0, LSE = -inf
                    if (row_on) {
#pragma unroll 1
                        for (int i = 0; i < D / 8; ++i) out[i] = make_uint4(0, 0, 0, 0);
                        p.lse[req * p.ls[0] + hq * p.ls[1] + tok] = -INFINITY;
                    }
                    continue;
                }
                // (an item on both chains has one pair of weights a row, posted by chain 0, and chain 1's barrier beside)
                ok = mbar_wait(bar(L::kWFull + c), (o_phase >> c) & 1u, ctx_item) &&
                     (!merge || mbar_wait(bar(L::kWFull + 1), (o_phase >> 1) & 1u, ctx_item));
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                const float wa = merge ? weight[2 * rloc] : weight[c * 128 + rloc];
                const float wb = merge ? weight[2 * rloc + 1] : 0.f;
                mbar_arrive(bar(L::kWEmpty + c));
                if (merge) mbar_arrive(bar(L::kWEmpty + 1));
                ok = mbar_wait(bar(L::kOFull + c), (o_phase >> c) & 1u, ctx_item) &&
                     (!merge || mbar_wait(bar(L::kOFull + 1), (o_phase >> 1) & 1u, ctx_item));
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                tc_fence_after_sync();
                const uint32_t t_c = t_o + c * D;
                if (quad * 32 >= nrow) {
                    // none of this warp's rows exist
                } else if (it.slot < 0) {
                    const bool zero = __float_as_uint(wa) == 0x80000000u;
#pragma unroll 1
                    for (int col = 0; col < D; col += 32) {
                        uint32_t o[32], pw[16];
                        tmem_ld32(t_c + col, o);
                        tmem_wait_ld(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * wa);
                        if (merge) {
                            // (a chain without a visible key for the row has weight 0 and finite O)
                            uint32_t ob[32];
                            tmem_ld32(t_c + D + col, ob);
                            tmem_wait_ld(ob);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = __float_as_uint(fmaf(__uint_as_float(ob[i]), wb, __uint_as_float(o[i])));
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            pw[i] = zero ? 0u : pack_bf16x2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
                        if (row_on) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                out[col / 8 + i] = make_uint4(pw[4 * i], pw[4 * i + 1], pw[4 * i + 2], pw[4 * i + 3]);
                        }
                    }
                } else {
                    // A piece, in fp32: by loads that give four threads 32 neighbouring bytes of a row.  Kept in L2
                    // (evict last): read back right after this grid.
                    const int ql = lane & 3, r4 = lane >> 2;
                    const uint64_t keep = l2_policy_evict_last();
                    const int here = nrow - quad * 32;  // rows of this warp
                    float* part = p.part_o + (static_cast<int64_t>(it.slot) * p.orows + k * p.qrows + quad * 32 + r4) * D + 2 * ql;
#pragma unroll 1
                    for (int half = 0; half < 32 && half < here; half += 16, part += 16 * D) {
                        const uint32_t t_h = t_c + (static_cast<uint32_t>(half) << 16);
                        const float wa0 = __shfl_sync(0xffffffffu, wa, half + r4), wa1 = __shfl_sync(0xffffffffu, wa, half + r4 + 8);
                        const float wb0 = __shfl_sync(0xffffffffu, wb, half + r4), wb1 = __shfl_sync(0xffffffffu, wb, half + r4 + 8);
#pragma unroll 1
                        for (int col = 0; col < D; col += 32) {
                            uint32_t oa[16];
                            tmem_ld16x256(t_h + col, oa);
                            tmem_wait_ld16(oa);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                oa[i] = __float_as_uint(__uint_as_float(oa[i]) * ((i & 2) ? wa1 : wa0));
                            if (merge) {
                                uint32_t ob[16];
                                tmem_ld16x256(t_h + D + col, ob);
                                tmem_wait_ld16(ob);
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    oa[i] = __float_as_uint(fmaf(__uint_as_float(ob[i]), (i & 2) ? wb1 : wb0, __uint_as_float(oa[i])));
                            }
#pragma unroll
                            for (int i = 0; i < 16; i += 4) {
                                if (half + r4 < here)
                                    st_global_v2_hint(part + col + 2 * i, __uint_as_float(oa[i]), __uint_as_float(oa[i + 1]), keep);
                                if (half + r4 + 8 < here)
                                    st_global_v2_hint(part + 8 * D + col + 2 * i, __uint_as_float(oa[i + 2]),
                                                      __uint_as_float(oa[i + 3]), keep);
                            }
                        }
                    }
                }
                tc_fence_before_sync();
                mbar_arrive(bar(L::kOEmpty + c));
                if (merge) mbar_arrive(bar(L::kOEmpty + 1));
            }
            if (nt > 0) {
                o_phase ^= two || merge ? 3u : 1u << par;
                par = two ? 0u : (par + nt) & 1u;
            }
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Merge the pieces of the units that stretches cut.  The cut units' rows are dealt to the warps of a grid that fills the GPU
// (a CTA for every stretch and row block, most of them with nothing to do, took 1.4 us for each thousand); where there
// are fewer rows than CTAs, the eight warps of a CTA share a row's pieces, each with a running maximum, and are merged in a
// fixed order.  Lane l holds columns [kPer l, kPer l + kPer).
constexpr int kPkMostStretches = 2048;

template <int D>
__global__ void __launch_bounds__(256, 4) attn_packed_combine_kernel(const __grid_constant__ PackedParams p) {
    constexpr int kPer = D / 32;
    __shared__ int s_first[kPkMostStretches + 1];  // rows of the cuts before each stretch's
    __shared__ int s_warp[8];
    __shared__ float s_acc[8][D];
    __shared__ float2 s_stat[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int carry = 0;
    for (int base = 0; base < p.stretches; base += 256) {
        const int i = base + threadIdx.x;
        int rows = 0;
        if (i < p.stretches) {
            const int* desc = reinterpret_cast<const int*>(p.cuts + i);
            rows = __ldcg(desc) > 0 ? __ldcg(desc + 4) : 0;
        }
        int sum = warp_scan(rows, lane);
        if (lane == 31) s_warp[warp] = sum;
        __syncthreads();
        int before = carry;
        for (int w = 0; w < 8; ++w) {
            if (w < warp) before += s_warp[w];
            carry += s_warp[w];
        }
        if (i < p.stretches) s_first[i] = before + sum - rows;
        __syncthreads();
    }
    const int total = carry;
    const bool shared = total <= static_cast<int>(gridDim.x);
    const int part = shared ? warp : 0, step = shared ? 8 : 1;
    for (int x = shared ? blockIdx.x : blockIdx.x * 8 + warp; x < total; x += shared ? gridDim.x : gridDim.x * 8) {
        int i = 0, end = p.stretches;  // the last stretch whose rows begin at or before x (it has some: the next begins after)
        while (end - i > 1) {
            const int mid = (i + end) / 2;
            if (s_first[mid] <= x) i = mid;
            else end = mid;
        }
        const int row = x - s_first[i];
        const int* desc = reinterpret_cast<const int*>(p.cuts + i);
        const int pieces = __ldcg(desc), head = __ldcg(desc + 1), req = __ldcg(desc + 2), tok0 = __ldcg(desc + 3);
        auto at = [&](int s) -> int64_t { return static_cast<int64_t>(s == 0 ? 2 * i + 1 : 2 * (i + s)) * p.orows + row; };
        float acc[kPer];
#pragma unroll
        for (int c = 0; c < kPer; ++c) acc[c] = 0.f;
        float sum = 0.f, mx = -INFINITY;
        constexpr int kUnroll = 4;
        for (int s0 = part; s0 < pieces; s0 += step * kUnroll) {
            float v[kUnroll][kPer], ls[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int s = s0 + u * step;
                ls[u] = -INFINITY;
#pragma unroll
                for (int c = 0; c < kPer; ++c) v[u][c] = 0.f;
                if (s < pieces) {
                    ls[u] = __ldcg(p.part_lse + at(s));
                    CombineVec<D>::load(p.part_o + at(s) * D + lane * kPer, v[u]);
                }
            }
            float m = mx;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) m = fmaxf(m, ls[u]);
            const float keep = mx == -INFINITY ? 0.f : expf(mx - m);
            mx = m;
            sum *= keep;
#pragma unroll
            for (int c = 0; c < kPer; ++c) acc[c] *= keep;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (ls[u] == -INFINITY) continue;  // no key of the piece is seen: what its row holds does not count
                const float w = expf(ls[u] - mx);
                sum += w;
#pragma unroll
                for (int c = 0; c < kPer; ++c) acc[c] = fmaf(w, v[u][c], acc[c]);
            }
        }
        if (shared) {
#pragma unroll
            for (int c = 0; c < kPer; ++c) s_acc[warp][lane * kPer + c] = acc[c];
            if (lane == 0) s_stat[warp] = make_float2(mx, sum);
            __syncthreads();
            if (warp == 0) {
                float m = mx;
                for (int k = 1; k < 8; ++k) m = fmaxf(m, s_stat[k].x);
                const float keep = mx == -INFINITY ? 1.f : expf(mx - m);  // (nothing yet, or a NaN to pass on)
                sum *= keep;
#pragma unroll
                for (int c = 0; c < kPer; ++c) acc[c] *= keep;
                for (int k = 1; k < 8; ++k) {
                    const float2 st = s_stat[k];
                    const float w = st.x == -INFINITY ? 1.f : expf(st.x - m);
                    sum += st.y * w;
#pragma unroll
                    for (int c = 0; c < kPer; ++c) acc[c] = fmaf(w, s_acc[k][lane * kPer + c], acc[c]);
                }
                mx = m;
            }
            __syncthreads();
        }
        if (part == 0) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const int t = row / p.G, hq = head * p.G + row - t * p.G;
            const int64_t r = p.lens ? req : 0, token = static_cast<int64_t>(tok0) + t;
            uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + r * p.os[0] + hq * p.os[1] + token * p.os[2] + lane * kPer);
#pragma unroll
            for (int c = 0; c < kPer; c += 2) dst[c / 2] = pack_bf16x2(acc[c] * inv, acc[c + 1] * inv);
            if (lane == 0) p.lse[r * p.ls[0] + hq * p.ls[1] + token] = sum == 0.f ? -INFINITY : mx + logf(sum);
        }
    }
}

}  // namespace elsattn
