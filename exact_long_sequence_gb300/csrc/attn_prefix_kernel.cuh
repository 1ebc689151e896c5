// Attention of a batch of requests that share a long prefix, for sm_103a: T new
// tokens of each of R requests against the prefix's keys and values (stored
// once) and the request's own.  Queries have Hq = G Hk heads; the G heads that
// share a key head, the T tokens and, for the prefix, all R requests are rows
// of one matrix, so the prefix costs one pass over its K/V (and one product
// with R G T rows), however many requests there are:
//     rows of key head h:  i = (r G + g) T + t,
//     O_i = sum_j p_ij V_j over the prefix's and r's own visible keys j.
// The two ranges (and pieces of them) are independent softmaxes, each giving
// O over its keys and its log-sum-exp; attn_prefix_combine_kernel merges them,
//     LSE = log sum_s exp(LSE_s),  O = sum_s exp(LSE_s - LSE) O_s,
// the combination step of the online softmax applied across pieces.
//
// A work item is (key head, up to 256 rows, a run of 128-key tiles of one K/V
// source).  One persistent CTA per SM runs the items of its share:
//   warp 0 (one lane)  TMA producer of K_j, V_j into a ring of stages
//   warp 1             tcgen05.mma issuer; owns the TMEM allocation
//   warp 2             scheduler: works out the CTA's items (the own lengths are
//                      device data) and passes them to the others through a ring
//   warp 3             Q loader: the rows of whole requests by TMA (a box of T x G x
//                      requests lands in row order), or row by row where a request has more than 128
//   warps 4-7, 8-11    softmax warpgroups, one per chain (below)
// Two chains (S_c, O_c in TMEM, softmax warpgroup c) alternate step by step, so
// that the tensor core works on one while the softmax of the other runs:
//   - an item of more than 128 rows has two query tiles, one a chain, that share
//     every K/V tile;
//   - an item of at most 128 rows has one query tile, and the chains take turns
//     with its K/V tiles (even tiles on one, odd on the other); their two
//     softmaxes are merged when the item ends, each warpgroup writing half of
//     the columns.
// The steps of consecutive items form one stream: the next item's first score
// product is issued before the last output product of this one, and an item of
// one query tile starts on the chain that the previous step left, so short
// items overlap too.
//
// What bounds it: up to about 128 rows a key head, reading K/V from HBM; with
// 256 and more, the tensor core (4 d operations a row and key).
#pragma once

#include <cuda.h>
#include <cstdint>
#include <type_traits>

#include "attn_fwd_kernel.cuh"
#include "plan.h"
#include "sm103_ptx.cuh"

namespace elsattn {

// Units of work: a tile of 128 keys is 4, a tail 1 for each 32 keys begun, an
// item besides its tiles (query rows, pipeline fill, epilogue) kPfxItemCost.
constexpr int kPfxTileCost = 4;
constexpr int kPfxItemCost = 2;
constexpr int kPfxOwnBox = 32;   // keys per TMA box of the own caches
constexpr int kPfxItemRing = 8;
constexpr int kOwnStep = 16;     // keys per step of the own-keys kernel

struct PrefixParams {
    const __nv_bfloat16* q;
    int64_t qs[3];          // strides in elements: request, head, token
    __nv_bfloat16* o;
    int64_t os[3];
    float* lse;             // [R, Hq, T]
    const int32_t* lens;    // [R] own keys, the new tokens among them (negative: padding); nullptr: none
    int R, T, Hk, G;
    int GT;                 // rows of a request at one key head
    int P, C;               // prefix keys; own capacity
    int qrows;              // rows of a query tile: the whole requests that fit 128 rows, or 128 if one does not
    int pblocks;            // blocks of two query tiles over R GT
    int ptiles;             // prefix tiles of a key head
    int psegs;              // stretches that the tiles are cut into (PrefixCut)
    int by_head;            // 1: each head is cut by itself, into psegs / Hk stretches; 0: the line of all heads is
    int run_len, run_per;   // tiles of a run (a head, or the line) and its stretches
    int even_base, even_rem;  // an even cut: run_per stretches of even_base tiles, the first even_rem one more
    int early;              // how many stretches of a run are longer, because their CTAs start before the others'; 0: an even cut
    int lead;               // how much longer: lead / 2^20 tiles for each step of own work
    int pitems;             // psegs * pblocks (a stretch at one row block)
    int oblocks;            // row blocks of a request at a key head, for its own keys,
    int orows;              // ... of so many rows: two query tiles, or up to 16 in the own-keys kernel (at most GT)
    float* part_o;          // partial rows [.., d] fp32: first [psegs + Hk - 1][R GT], then [own slots][orows]
    float* part_lse;        // one per partial row
    int64_t own_first;      // the first own slot's partial row
    int* own_start;         // [R + 1]: where each request's own work starts, and the total
    int workers;            // warps of attn_prefix_own_kernel, which then does the own work; 0: it is items of the prefix kernel
    uint32_t* error_word;
    uint64_t timeout_ns;
    float scale_log2, max_scale_log2;
    uint32_t negate_scores;
};

// Own work is laid on a line: request by request, its (key head, row block)
// sequences in order, each kPfxItemCost units and then its tiles.  The line is
// cut into one stretch per CTA: CTAs [0, rem) have one prefix item more than
// the others and get cap1 units, the others cap0, so that all end together.
// A tile belongs to the CTA whose stretch holds the tile's first unit.  Caps
// are 0 or at least a tile, so every CTA between the first and the last of a
// sequence has a tile of it.
// (All counts of work fit 32 bits: the host refuses shapes whose do not.)
struct OwnCut {
    int rem, cap1, cap0;
    __device__ __forceinline__ OwnCut(const PrefixParams& p, int total, int grid) {
        rem = p.pitems % grid;
        // (with own items the stretches are even: at most this many tiles)
        const int item = p.psegs == 0 ? 0 : kPfxItemCost + (p.Hk * p.ptiles + p.psegs - 1) / p.psegs * kPfxTileCost;
        const int64_t level = static_cast<int64_t>(item) * (grid - rem);  // what evens the CTAs out
        if (rem == 0 || total > level) {
            const int e = (total - (rem == 0 ? 0 : static_cast<int>(level)) + grid - 1) / grid;
            cap1 = e;
            cap0 = rem == 0 ? e : item + e;
        } else {
            cap1 = 0;
            cap0 = (total + grid - rem - 1) / (grid - rem);
        }
        if (cap1 > 0 && cap1 < kPfxTileCost) cap1 = kPfxTileCost;
        if (cap0 < kPfxTileCost) cap0 = kPfxTileCost;
    }
    // (the last stretches may begin past the line's end, and past 32 bits)
    __device__ __forceinline__ int64_t begin(int cta) const {
        return cta < rem ? static_cast<int64_t>(cta) * cap1
                         : static_cast<int64_t>(rem) * cap1 + static_cast<int64_t>(cta - rem) * cap0;
    }
    __device__ __forceinline__ int cta_of(int x) const {
        return x < rem * cap1 ? x / cap1 : rem + (x - rem * cap1) / cap0;
    }
};
__device__ __forceinline__ int own_len(const PrefixParams& p, int r) { return min(max(__ldg(p.lens + r), 0), p.C); }
// Units of one sequence of a request with `len` own keys (0: no work), and of the request.
__device__ __forceinline__ int seq_cost(int len) { return len > 0 ? kPfxItemCost + (len + 31) / 32 : 0; }
__device__ __forceinline__ int request_cost(const PrefixParams& p, int len) { return seq_cost(len) * (p.Hk * p.oblocks); }

// Units of one sequence in the own-keys kernel (WarpCut).
__device__ __forceinline__ int warp_seq_cost(int len) { return len > 0 ? 1 + (len + kOwnStep - 1) / kOwnStep : 0; }

// Inclusive sum over the warp's lanes.
__device__ __forceinline__ int warp_scan(int v, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += o;
    }
    return v;
}

// The cut of the prefix's tiles.  Where the number of stretches allows it each
// key head is cut by itself (the stretches go head by head, first all early
// ones, then the others); otherwise the line of all heads' tiles is, and a
// stretch may cross heads.  A stretch's tiles at one head are a piece.  The row blocks of a stretch are
// neighbouring items, which run at the same time and share its K/V in L2.
// The stretches are even, but where the own keys' kernel holds many SMs: the
// CTAs of the first stretches start beside it, the others after it, so the
// first are longer by its time in tiles.
struct PrefixCut {
    int len, per;           // tiles of a run (a head, or the line), and its stretches
    int etiles, ebase, erem;  // the early stretches' tiles; each has ebase, the first erem one more
    int lbase, lrem;        // the others'
    __device__ __forceinline__ PrefixCut(const PrefixParams& p, int own_total)
        : len(p.run_len), per(p.run_per), etiles(0), ebase(0), erem(0), lbase(p.even_base), lrem(p.even_rem) {
        if (p.early == 0) return;
        // early ones `delta` longer: per * late + early * delta = len, late >= 0  (0 < early < per <= len)
        const int64_t delta = (static_cast<int64_t>(own_total) * p.lead) >> 20;
        const int64_t ahead = min(static_cast<int64_t>(len), p.early * delta);
        const int late = (len - static_cast<int>(ahead)) / per;
        etiles = len - late * (per - p.early);
        ebase = etiles / p.early;
        erem = etiles - ebase * p.early;
        lbase = late;  // what is left over is the early ones'
        lrem = 0;
    }
    __device__ __forceinline__ int run_begin(const PrefixParams& p, int i) const {
        return i < p.early ? i * ebase + min(i, erem) : etiles + (i - p.early) * lbase + min(i - p.early, lrem);
    }
    // Stretch k as the i-th of a run (of head `run`, or of the line).
    __device__ __forceinline__ void place(const PrefixParams& p, int k, int& run, int& i) const {
        run = 0;
        i = k;
        if (!p.by_head) return;
        const int first = p.early * p.Hk, n = k < first ? p.early : per - p.early;
        const int y = k < first ? k : k - first;
        run = y / n;
        i = y - run * n + (k < first ? 0 : p.early);
    }
    // The stretch of a run that tile y of it is in.
    __device__ __forceinline__ int run_of(const PrefixParams& p, int y) const {
        if (y < etiles) {
            const int longer = erem * (ebase + 1);
            return y < longer ? y / (ebase + 1) : erem + (y - longer) / ebase;
        }
        y -= etiles;
        const int longer = lrem * (lbase + 1);
        return p.early + (y < longer ? y / (lbase + 1) : lrem + (y - longer) / lbase);
    }
    // Partial rows of the piece of a run's i-th stretch at a head (the row blocks are parts of them).  In the
    // line, pieces in order step to the next stretch or to the next head, so that their sum numbers them apart.
    __device__ __forceinline__ int64_t part(const PrefixParams& p, int i, int head) const {
        return static_cast<int64_t>(p.by_head ? head * per + i : i + head) * p.R * p.GT;
    }
};

struct PrefixItem {
    int ntiles;      // -1: no more items
    int tile0;       // first tile
    int klen;        // keys of the source (the own length, or P)
    int head;        // key head
    int req;         // request of an own item; -1: the prefix
    int row0, nrows; // rows of the key head's matrix
    int pad;
    int64_t part;    // partial row of row0
};

template <int D>
struct PrefixSmem {
    static constexpr int kTile = tile_bytes(D);
    static constexpr int kStages = kv_stages_for(D);
    static constexpr int kQOff = 0;
    static constexpr int kRingOff = kQTiles * kTile;
    static constexpr int kXchgOff = kRingOff + kStages * kTile;   // [128] (m, l) of one chain, then of the other
    static constexpr int kItemOff = kXchgOff + 128 * 8;           // [kPfxItemRing] PrefixItem
    static constexpr int kBarOff = kItemOff + kPfxItemRing * static_cast<int>(sizeof(PrefixItem));
    static constexpr int kKvFull = 0;
    static constexpr int kKvEmpty = kKvFull + kStages;
    static constexpr int kQFull = kKvEmpty + kStages;     // [2] by slot
    static constexpr int kQEmpty = kQFull + 2;            // [2]
    static constexpr int kSFull = kQEmpty + 2;            // [2] by chain, as all below
    static constexpr int kPHalf = kSFull + 2;             // [2] first half of P stored, O rescaled
    static constexpr int kPFull = kPHalf + 2;             // [2]
    static constexpr int kOFull = kPFull + 2;             // [2]
    static constexpr int kOEmpty = kOFull + 2;            // [2]
    static constexpr int kX = kOEmpty + 2;                // [2] the chain's (m, l) are in shared memory
    static constexpr int kDrain = kX + 2;
    static constexpr int kItemFull = kDrain + 1;          // [kPfxItemRing]
    static constexpr int kItemEmpty = kItemFull + kPfxItemRing;
    static constexpr int kNumBars = kItemEmpty + kPfxItemRing;
    static constexpr int kFlagsOff = kBarOff + kNumBars * 8;
    static constexpr int kBytes = kFlagsOff + 16 + kSmemAlign;
    static_assert(sizeof(PrefixItem) % 8 == 0, "barriers are 8-byte aligned");
    static_assert(kBytes <= kSmemLimit, "shared memory");
    static_assert(2 * kBytes > 233472, "one CTA per SM (each allocates all of TMEM)");
};
constexpr int kPfxItemReaders = 11;  // producer, MMA, Q loader, eight softmax warps

// 4-D and 5-D tiled loads.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void* tmap, uint32_t bar, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3, int32_t c4) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, uint32_t bar, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}
// 16 TMEM lanes x 32 columns: thread i of the warp gets, for each block of 8
// columns b, columns 2 (i % 4), 2 (i % 4) + 1 of lane i / 4 in r[4 b], r[4 b + 1]
// and of lane i / 4 + 8 in r[4 b + 2], r[4 b + 3]; four threads hold 32
// neighbouring bytes of a row, so a store fills whole sectors.
__device__ __forceinline__ void tmem_ld16x256(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void st_global_v2_hint(float* p, float a, float b, uint64_t pol) {
    asm volatile("st.global.L2::cache_hint.v2.f32 [%0], {%1, %2}, %3;" ::"l"(p), "f"(a), "f"(b), "l"(pol) : "memory");
}
// Whether the phase with the given parity has completed; never waits.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_prefix_kernel(const __grid_constant__ CUtensorMap tmap_qp, const __grid_constant__ CUtensorMap tmap_qo,
                   const __grid_constant__ CUtensorMap tmap_kp, const __grid_constant__ CUtensorMap tmap_vp,
                   const __grid_constant__ CUtensorMap tmap_ko, const __grid_constant__ CUtensorMap tmap_vo,
                   const __grid_constant__ PrefixParams p) {
    using L = PrefixSmem<D>;
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

    if (threadIdx.x == 0) {
        *abort_flag = 0u;
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(bar(L::kKvFull + s), 1);
            mbar_init(bar(L::kKvEmpty + s), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(L::kQFull + t), 32);
            mbar_init(bar(L::kQEmpty + t), 1);
            mbar_init(bar(L::kSFull + t), 1);
            mbar_init(bar(L::kPHalf + t), 128);
            mbar_init(bar(L::kPFull + t), 128);
            mbar_init(bar(L::kOFull + t), 1);
            mbar_init(bar(L::kOEmpty + t), 256);  // both warpgroups, or one that counts twice
            mbar_init(bar(L::kX + t), 128);
        }
        mbar_init(bar(L::kDrain), 1);
        for (int s = 0; s < kPfxItemRing; ++s) {
            mbar_init(bar(L::kItemFull + s), 1);
            mbar_init(bar(L::kItemEmpty + s), kPfxItemReaders);
        }
        fence_barrier_init();
        if (p.GT <= kBr) {
            tma_prefetch_desc(p.P > 0 ? &tmap_qp : &tmap_qo);
        }
        if (p.P > 0) {
            tma_prefetch_desc(&tmap_kp);
            tma_prefetch_desc(&tmap_vp);
        }
        if (p.C > 0 && p.workers == 0) {
            tma_prefetch_desc(&tmap_ko);
            tma_prefetch_desc(&tmap_vo);
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
    // The combine kernel may be scheduled onto SMs as this grid's CTAs retire;
    // it waits for the whole grid before it reads the partial results.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // Reads the next item (ring entry n); `it.ntiles` is -1 after the last.
    // Called by whole warps, or by one lane (whole = false).  keep: the caller
    // gives the ring entry back itself (the softmax warps read it again at the item's end).
    auto take_item = [&](uint32_t n, PrefixItem& it, bool whole, bool keep = false) -> bool {
        const uint32_t s = n % kPfxItemRing;
        bool got = mbar_wait(bar(L::kItemFull + s), (n / kPfxItemRing) & 1u, ctx);
        if (whole) got = __all_sync(0xffffffffu, got);
        if (!got) return false;
        const int* from = reinterpret_cast<const int*>(smem + L::kItemOff + s * sizeof(PrefixItem));
        if (whole) {
            // one word a lane, handed round by shuffles: the compiler then knows the fields to be the
            // same for the whole warp and keeps what follows from them in uniform registers
            const int word = from[lane < static_cast<int>(sizeof(PrefixItem) / 4) ? lane : 0];
            it.ntiles = __shfl_sync(0xffffffffu, word, 0);
            it.tile0 = __shfl_sync(0xffffffffu, word, 1);
            it.klen = __shfl_sync(0xffffffffu, word, 2);
            it.head = __shfl_sync(0xffffffffu, word, 3);
            it.req = __shfl_sync(0xffffffffu, word, 4);
            it.row0 = __shfl_sync(0xffffffffu, word, 5);
            it.nrows = __shfl_sync(0xffffffffu, word, 6);
            const uint32_t lo = __shfl_sync(0xffffffffu, word, 8), hi = __shfl_sync(0xffffffffu, word, 9);
            it.part = static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo);
        } else {
            it = *reinterpret_cast<const PrefixItem*>(from);
        }
        if (!keep && (!whole || lane == 0)) mbar_arrive(bar(L::kItemEmpty + s));
        return it.ntiles >= 0;
    };
    // Keys of the item's tile j (1 .. 128).
    auto tile_keys = [](const PrefixItem& it, int j) -> int { return min(kBc, it.klen - (it.tile0 + j) * kBc); };

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            RingPos pos{0u, 0u};
            uint32_t issued = 0;
            bool ok = true;
            PrefixItem it;
            for (uint32_t n = 0; ok && take_item(n, it, false); ++n) {
                for (int j = 0; j < it.ntiles && ok; ++j) {
                    const int key = (it.tile0 + j) * kBc;
                    const int boxes = (tile_keys(it, j) + kPfxOwnBox - 1) / kPfxOwnBox;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        ok = mbar_wait(bar(L::kKvEmpty + pos.stage), pos.phase ^ 1u, ctx);
                        if (!ok) break;
                        const uint32_t full = bar(L::kKvFull + pos.stage);
                        const uint32_t dst = s_base + L::kRingOff + pos.stage * L::kTile;
                        if (it.req < 0) {
                            mbar_arrive_expect_tx(full, L::kTile);
#pragma unroll
                            for (int b = 0; b < D / 64; ++b)
                                tma_load_3d(dst + b * (kBc * 128), kv == 0 ? &tmap_kp : &tmap_vp, full, b * 64, key,
                                            it.head);
                        } else {
                            mbar_arrive_expect_tx(full, boxes * kPfxOwnBox * D * 2);
                            for (int i = 0; i < boxes; ++i)
#pragma unroll
                                for (int b = 0; b < D / 64; ++b)
                                    tma_load_4d(dst + b * (kBc * 128) + i * (kPfxOwnBox * 128),
                                                kv == 0 ? &tmap_ko : &tmap_vo, full, b * 64, key + i * kPfxOwnBox,
                                                it.head, it.req);
                        }
                        pos = pos.next(L::kStages);
                        ++issued;
                    }
                }
            }
            // every issued copy lands before the CTA's shared memory is released (bounded waits)
            const uint32_t pending = issued < static_cast<uint32_t>(L::kStages) ? issued : L::kStages;
            RingPos back = pos;
            for (uint32_t i = 0; i < pending; ++i) {
                back = back.stage == 0 ? RingPos{L::kStages - 1u, back.phase ^ 1u} : RingPos{back.stage - 1, back.phase};
                mbar_wait_drain(bar(L::kKvFull + back.stage), back.phase, 50000000ull);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        const uint32_t idesc_s = make_idesc_bf16_f32(kBr, kBc, false, false) | (p.negate_scores ? kIdescNegateB : 0u);
        constexpr uint32_t idesc_o = make_idesc_bf16_f32(kBr, D, false, true);
        const uint64_t dq0 = make_smem_desc_sw128(s_base + L::kQOff, 16, 1024);
        const uint64_t dk0 = make_smem_desc_sw128(s_base + L::kRingOff, 16, 1024);
        const uint64_t dv0 = make_smem_desc_sw128(s_base + L::kRingOff, kBc * 128, 1024);
        uint32_t p_phase = 0u, o_phase = 3u;  // parities to wait for, bit c of chain c
        RingPos kpos{0u, 0u};   // K of the current tile
        uint32_t qpos = 0;      // query tiles taken so far: slot qpos & 1
        uint32_t par = 0;       // chain of the item's first step
        bool ok = true;
        // S_c = Q K^T, the operands' descriptors given
        auto gemm_s = [&](int c, uint64_t a, uint64_t b) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t off = static_cast<uint64_t>(((kk >> 2) * (kBr * 128) + (kk & 3) * 32) >> 4);
                mma_ss(tmem + c * kBc, a + off, b + off, idesc_s, kk > 0 ? 1u : 0u);
            }
        };
        // the output product that is due: of the step before
        struct { bool due, first, last, first_v, last_v; int chain, ksteps; RingPos v; } pv{};
        auto run_pv = [&]() -> bool {
            if (!pv.due) return true;
            pv.due = false;
            const int c = pv.chain;
            bool w = true;
            if (pv.first_v) w = mbar_wait(bar(L::kKvFull + pv.v.stage), pv.v.phase, ctx);
            w = w && mbar_wait(bar(L::kPHalf + c), (p_phase >> c) & 1u, ctx);
            if (pv.first) {
                w = w && mbar_wait(bar(L::kOEmpty + c), (o_phase >> c) & 1u, ctx);
                o_phase ^= 1u << c;
            }
            if (!__all_sync(0xffffffffu, w)) return false;
            tc_fence_after_sync();
            const uint64_t b = dv0 + static_cast<uint64_t>((pv.v.stage * L::kTile) >> 4);
            // products over keys [64 half, 64 half + 64), in steps of 16 up to the tile's last key
            auto gemm_o = [&](int half) {
#pragma unroll
                for (int kk = half * 4; kk < half * 4 + 4; ++kk)
                    if (kk < pv.ksteps)
                        mma_ts(tmem + 2 * kBc + c * D, tmem + c * kBc + kk * 8,
                               b + static_cast<uint64_t>((kk * 16 * 128) >> 4), idesc_o, (!pv.first || kk > 0) ? 1u : 0u);
            };
            if (elect_one()) gemm_o(0);
            __syncwarp();
            w = mbar_wait(bar(L::kPFull + c), (p_phase >> c) & 1u, ctx);
            p_phase ^= 1u << c;
            if (!__all_sync(0xffffffffu, w)) return false;
            tc_fence_after_sync();
            if (elect_one()) {
                gemm_o(1);
                if (pv.last_v) mma_commit(bar(L::kKvEmpty + pv.v.stage));
                if (pv.last) mma_commit(bar(L::kOFull + c));
            }
            __syncwarp();
            return true;
        };
        // The next score product goes first where its operands are there already: the tensor core
        // works on it while the softmax of the step before runs.  Where they are not (short items,
        // the ends of a CTA's share), the product that is due does not wait for them.
        auto there = [&](uint32_t b, uint32_t parity) -> bool { return __all_sync(0xffffffffu, mbar_test(b, parity)); };
        PrefixItem it;
        for (uint32_t n = 0; ok; ++n) {
            if (pv.due && !there(bar(L::kItemFull + n % kPfxItemRing), (n / kPfxItemRing) & 1u) && !(ok = run_pv())) break;
            if (!take_item(n, it, true)) break;
            const int nt = it.ntiles;
            if (it.nrows > p.qrows) {
                // Two query tiles, chain = tile: S0_j; O1 += P1_{j-1} V_{j-1}; S1_j; O0 += P0_j V_j.
                // The chains are literal in this loop, which is what bounds it: the issue of
                // a step's products and its waits, with generic steps, took 1.2 us.
                const uint32_t q0 = qpos & 1u, q1 = q0 ^ 1u;
                if (pv.due && (pv.chain == 0 || !there(bar(L::kKvFull + kpos.stage), kpos.phase) ||
                               !there(bar(L::kQFull + q0), (qpos >> 1) & 1u)) && !(ok = run_pv()))
                    break;
                const uint64_t a0 = dq0 + static_cast<uint64_t>((q0 * L::kTile) >> 4);
                const uint64_t a1 = dq0 + static_cast<uint64_t>((q1 * L::kTile) >> 4);
                const int last_steps = (tile_keys(it, nt - 1) + 15) / 16;
                // O_c (+)= P_c V_j, V_j at ring position v
                auto pv_two = [&](auto chain, int j, RingPos v) -> bool {
                    constexpr int c = decltype(chain)::value;
                    bool w = true;
                    if (c == 0) w = mbar_wait(bar(L::kKvFull + v.stage), v.phase, ctx);
                    w = w && mbar_wait(bar(L::kPHalf + c), (p_phase >> c) & 1u, ctx);
                    if (j == 0) {
                        w = w && mbar_wait(bar(L::kOEmpty + c), (o_phase >> c) & 1u, ctx);
                        o_phase ^= 1u << c;
                    }
                    if (!__all_sync(0xffffffffu, w)) return false;
                    tc_fence_after_sync();
                    const uint64_t b = dv0 + static_cast<uint64_t>((v.stage * L::kTile) >> 4);
                    const int ks = j == nt - 1 ? last_steps : kBc / 16;
                    auto gemm = [&](int half) {
#pragma unroll
                        for (int kk = half * 4; kk < half * 4 + 4; ++kk)
                            if (kk < ks)
                                mma_ts(tmem + 2 * kBc + c * D, tmem + c * kBc + kk * 8,
                                       b + static_cast<uint64_t>((kk * 16 * 128) >> 4), idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
                    };
                    if (elect_one()) gemm(0);
                    __syncwarp();
                    w = mbar_wait(bar(L::kPFull + c), (p_phase >> c) & 1u, ctx);
                    p_phase ^= 1u << c;
                    if (!__all_sync(0xffffffffu, w)) return false;
                    tc_fence_after_sync();
                    if (elect_one()) {
                        gemm(1);
                        if (c == 1) mma_commit(bar(L::kKvEmpty + v.stage));
                        if (j == nt - 1) mma_commit(bar(L::kOFull + c));
                    }
                    __syncwarp();
                    return true;
                };
                RingPos vprev{0u, 0u};
                for (int j = 0; j < nt && ok; ++j) {
                    bool w = mbar_wait(bar(L::kKvFull + kpos.stage), kpos.phase, ctx);
                    if (j == 0)
                        w = w && mbar_wait(bar(L::kQFull + q0), (qpos >> 1) & 1u, ctx) &&
                            mbar_wait(bar(L::kQFull + q1), ((qpos + 1) >> 1) & 1u, ctx);
                    if (!(ok = __all_sync(0xffffffffu, w))) break;
                    const uint64_t b = dk0 + static_cast<uint64_t>((kpos.stage * L::kTile) >> 4);
                    if (elect_one()) {
                        gemm_s(0, a0, b);
                        mma_commit(bar(L::kSFull + 0));
                        if (j == nt - 1) mma_commit(bar(L::kQEmpty + q0));
                    }
                    __syncwarp();
                    ok = j == 0 ? run_pv() : pv_two(std::integral_constant<int, 1>{}, j - 1, vprev);
                    if (!ok) break;
                    if (elect_one()) {
                        gemm_s(1, a1, b);
                        mma_commit(bar(L::kSFull + 1));
                        mma_commit(bar(L::kKvEmpty + kpos.stage));
                        if (j == nt - 1) mma_commit(bar(L::kQEmpty + q1));
                    }
                    __syncwarp();
                    vprev = kpos.next(L::kStages);
                    if (!(ok = pv_two(std::integral_constant<int, 0>{}, j, vprev))) break;
                    kpos = vprev.next(L::kStages);
                }
                if (!ok) break;
                pv.due = true;
                pv.chain = 1;
                pv.v = vprev;
                pv.ksteps = last_steps;
                pv.first = nt == 1;
                pv.last = true;
                pv.first_v = false;
                pv.last_v = true;
                qpos += 2;
                par = 0;
                continue;
            }
            // One query tile; the chains take turns with the K/V tiles.
            const uint32_t qslot = qpos & 1u;
            for (int j = 0; j < nt && ok; ++j) {
                const int c = (par + j) & 1;
                if (pv.due && (!there(bar(L::kKvFull + kpos.stage), kpos.phase) ||
                               (j == 0 && !there(bar(L::kQFull + qslot), (qpos >> 1) & 1u))) && !(ok = run_pv()))
                    break;
                bool w = mbar_wait(bar(L::kKvFull + kpos.stage), kpos.phase, ctx);
                if (j == 0) w = w && mbar_wait(bar(L::kQFull + qslot), (qpos >> 1) & 1u, ctx);
                if (!(ok = __all_sync(0xffffffffu, w))) break;
                if (elect_one()) {
                    gemm_s(c, dq0 + static_cast<uint64_t>((qslot * L::kTile) >> 4),
                           dk0 + static_cast<uint64_t>((kpos.stage * L::kTile) >> 4));
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
        auto publish = [&](const PrefixItem& it) {
            const uint32_t s = n % kPfxItemRing;
            if (n >= kPfxItemRing) ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kItemEmpty + s), ((n / kPfxItemRing) - 1) & 1u, ctx));
            if (!ok) return;
            if (lane == 0) {
                *reinterpret_cast<PrefixItem*>(smem + L::kItemOff + s * sizeof(PrefixItem)) = it;
                mbar_arrive(bar(L::kItemFull + s));
            }
            __syncwarp();
            ++n;
        };
        PrefixItem it;
        it.pad = 0;
        int own_total = 0;
        if (p.early > 0) {  // (with the own-keys kernel)
#pragma unroll 4
            for (int r = lane; r < p.R; r += 32) own_total += warp_seq_cost(own_len(p, r));
            own_total = __reduce_add_sync(0xffffffffu, own_total) * (p.Hk * p.oblocks);
        }
        const PrefixCut cut(p, own_total);
        for (int i = blockIdx.x; i < p.pitems && ok; i += gridDim.x) {
            const int blk = i % p.pblocks, k = i / p.pblocks;
            it.req = -1;
            it.klen = p.P;
            it.row0 = blk * 2 * p.qrows;
            it.nrows = min(2 * p.qrows, p.R * p.GT - it.row0);
            int run, nth;
            cut.place(p, k, run, nth);
            const int base = run * cut.len, end = base + cut.run_begin(p, nth + 1);
            for (int x = base + cut.run_begin(p, nth); x < end && ok; x += it.ntiles) {
                it.head = x / p.ptiles;
                it.tile0 = x - it.head * p.ptiles;
                it.ntiles = min(end - x, p.ptiles - it.tile0);
                it.part = cut.part(p, nth, it.head) + it.row0;
                publish(it);
            }
        }
        if (p.C > 0 && p.workers == 0 && ok) {
            // The total and the lane whose run of requests holds this CTA's first unit.
            const int run = (p.R + 31) / 32;
            int mine = 0;
#pragma unroll 8
            for (int i = 0; i < run; ++i) {
                const int r = lane * run + i;
                mine += seq_cost(r < p.R ? own_len(p, r) : 0);
            }
            mine *= p.Hk * p.oblocks;
            const int upto = warp_scan(mine, lane);
            const int total = __shfl_sync(0xffffffffu, upto, 31);
            const OwnCut own(p, total, gridDim.x);
            const int x0 = static_cast<int>(min(own.begin(blockIdx.x), static_cast<int64_t>(total)));
            const int x1 = static_cast<int>(min(own.begin(blockIdx.x + 1), static_cast<int64_t>(total)));
            if (x0 < x1) {
                const int at = __ffs(__ballot_sync(0xffffffffu, upto > x0)) - 1;
                int start = __shfl_sync(0xffffffffu, upto - mine, at);  // of request r0
                for (int r0 = at * run; r0 < p.R && start < x1 && ok; r0 += 32) {
                    const int len_l = r0 + lane < p.R ? own_len(p, r0 + lane) : 0;
                    for (int i = 0; i < 32 && start < x1 && ok; ++i) {
                        const int len = __shfl_sync(0xffffffffu, len_l, i);
                        const int cost = seq_cost(len);
                        const int seqs = p.Hk * p.oblocks;
                        if (len > 0 && start + cost * seqs > x0) {
                            const int nt = (len + kBc - 1) / kBc;
                            int q = x0 > start ? (x0 - start) / cost : 0;
                            for (; q < seqs && start + q * cost < x1 && ok; ++q) {
                                const int first = start + q * cost + kPfxItemCost;  // tile 0's unit
                                const int a = x0 > first ? (x0 - first + kPfxTileCost - 1) / kPfxTileCost : 0;
                                const int b = x1 > first ? (x1 - first + kPfxTileCost - 1) / kPfxTileCost : 0;
                                const int t0 = min(a, nt);
                                const int t1 = min(b, nt);
                                if (t0 >= t1) continue;
                                const int blk = q % p.oblocks;
                                it.head = q / p.oblocks;
                                it.req = r0 + i;
                                it.klen = len;
                                it.tile0 = t0;
                                it.ntiles = t1 - t0;
                                it.row0 = it.req * p.GT + blk * 2 * p.qrows;
                                it.nrows = min(2 * p.qrows, p.GT - blk * 2 * p.qrows);
                                const int64_t slot = (static_cast<int64_t>(it.req) * p.Hk * p.oblocks + q) + blockIdx.x;
                                it.part = p.own_first + slot * p.orows;
                                publish(it);
                            }
                        }
                        start += cost * seqs;
                    }
                }
            }
        }
        it.ntiles = -1;
        if (ok) publish(it);
        // One CTA leaves every request's start and the total for the combine kernel.
        if (p.C > 0 && p.workers == 0 && blockIdx.x == gridDim.x - 1) {
            int start = 0;
            for (int r0 = 0; r0 < p.R; r0 += 32) {
                const int c = r0 + lane < p.R ? request_cost(p, own_len(p, r0 + lane)) : 0;
                const int upto = warp_scan(c, lane);
                if (r0 + lane < p.R) p.own_start[r0 + lane] = start + upto - c;
                start += __shfl_sync(0xffffffffu, upto, 31);
            }
            if (lane == 0) p.own_start[p.R] = start;
        }
    } else if (warp == 3) {
        // ------------------------------------------------------------ Q loader
        constexpr int kChunks = D / 8;            // 16-byte chunks of a row
        constexpr int kRows = 32 / kChunks;       // rows per pass of the warp
        const int ch = lane % kChunks, sub = lane / kChunks;
        const uint32_t col = (ch >> 3) * (kBr * 128);
        uint32_t qpos = 0;
        uint32_t q_slots = 0, q_parity = 0;  // slots that a TMA copy was issued to, and the parity it completes
        bool ok = true;
        PrefixItem it;
        for (uint32_t n = 0; ok && take_item(n, it, true); ++n) {
            for (int k = 0; k < (it.nrows > p.qrows ? 2 : 1) && ok; ++k, ++qpos) {
                const uint32_t slot = qpos & 1u;
                ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kQEmpty + slot), ((qpos >> 1) & 1u) ^ 1u, ctx));
                if (!ok) break;
                if (p.GT <= kBr) {
                    // whole requests: those of the tile (past the last they read as zero), or the item's own
                    const uint32_t full = bar(L::kQFull + slot);
                    if (lane == 0) {
                        const int rows = it.req < 0 ? p.qrows : p.GT;
                        mbar_arrive_expect_tx(full, rows * D * 2);
#pragma unroll
                        for (int b = 0; b < D / 64; ++b)
                            tma_load_5d(s_base + L::kQOff + slot * L::kTile + b * (kBr * 128),
                                        it.req < 0 ? &tmap_qp : &tmap_qo, full, b * 64, 0, 0, it.head,
                                        (it.row0 + k * p.qrows) / p.GT);
                        q_slots |= 1u << slot;
                        q_parity = (q_parity & ~(1u << slot)) | (((qpos >> 1) & 1u) << slot);
                    } else {
                        mbar_arrive(full);
                    }
                    __syncwarp();
                    continue;
                }
                const int rows = min(kBr, it.nrows - k * kBr);
                const uint32_t dst = s_base + L::kQOff + slot * L::kTile + col;
                for (int base = 0; base < rows; base += 32) {
                    // lane l works out where row base + l is
                    const int row = it.row0 + k * kBr + min(base + lane, rows - 1);
                    const int r = row / p.GT, x = row - r * p.GT;
                    const int g = x / p.T, t = x - g * p.T;
                    const int64_t at = r * p.qs[0] + (static_cast<int64_t>(it.head) * p.G + g) * p.qs[1] + t * p.qs[2];
                    for (int i0 = 0; i0 < 32 && base + i0 < rows; i0 += 4 * kRows) {
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const int i = i0 + u * kRows + sub;
                            const int64_t from = __shfl_sync(0xffffffffu, at, i);
                            const int rr = base + i;
                            if (rr < rows)
                                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                                 dst + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4)),
                                             "l"(p.q + from + ch * 8)
                                             : "memory");
                        }
                    }
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                fence_proxy_async_smem();
                mbar_arrive(bar(L::kQFull + slot));
            }
        }
        for (uint32_t s = 0; s < 2; ++s)  // the copies land before the shared memory is released
            if (q_slots & (1u << s)) mbar_wait_drain(bar(L::kQFull + s), (q_parity >> s) & 1u, 50000000ull);
    } else {
        // ------------------------------------------------------------ softmax warpgroups
        const int t = (warp - 4) >> 2;          // chain
        const int quad = warp & 3;              // TMEM lane quadrant
        const int rloc = quad * 32 + lane;      // row within the tile
        const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t t_s = tmem + lane_addr + t * kBc;
        const uint32_t t_o = tmem + lane_addr + 2 * kBc;  // O_0; O_1 is D columns further
        float2* xchg = reinterpret_cast<float2*>(smem + L::kXchgOff);
        const float sl2 = p.scale_log2;
        uint32_t s_cnt = 0, x_cnt = 0, ring = 0;  // ring: K/V fills before this item
        uint32_t o_phase = 0u;                    // parity of each chain's next finished item, bit c
        uint32_t par = 0;
        bool ok = true;
        PrefixItem it;
        for (uint32_t n = 0; ok && take_item(n, it, true, true); ++n) {
            const bool two = it.nrows > p.qrows;
            const int nt = it.ntiles;
            const bool own = it.req >= 0;
            const int mine = two ? t : t ^ static_cast<int>(par);  // this chain's query tile, or its first K/V tile
            const int k = two ? mine : 0;                     // its query tile
            const int nrow = min(p.qrows, it.nrows - k * p.qrows);
            const bool warp_on = quad * 32 < nrow;            // the warp has rows
            const bool row_on = rloc < nrow;
            const bool both = two || nt >= 2;                 // both chains work on the item
            const bool used = both || mine == 0;
            float m_ref = -INFINITY;
            float l = 0.f;
            if (used) {
                // Key counts from the item's first tile on: all of the source's, and those that this row
                // sees (not the later tokens' of its own request) and every row does.
                const int left = it.klen - it.tile0 * kBc;
                int lim = left;
                if (own && p.T > 1) {
                    const int x = it.row0 + k * p.qrows + min(rloc, nrow - 1) - it.req * p.GT;
                    lim -= p.T - 1 - x % p.T;
                }
                const int all_see = left - (own ? p.T - 1 : 0);
                bool first = true;
                for (int j = two ? 0 : mine; j < nt; j += two ? 1 : 2) {
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kSFull + t), s_cnt & 1u, ctx));
                    ++s_cnt;
                    if (!ok) break;
                    tc_fence_after_sync();
                    const int key0 = j * kBc;
                    const int keys = min(kBc, left - key0);
                    // The output product sums over keys in steps of 16.  Own-cache rows past the
                    // last key may hold anything (a NaN times a zero weight is a NaN): zero them.
                    if (own && k == 0 && (keys & 15) != 0) {
                        const uint32_t at = ring + 2 * j + 1;  // V_j's fill
                        const uint32_t stage = at % L::kStages;
                        ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kKvFull + stage), (at / L::kStages) & 1u, ctx));
                        if (!ok) break;
                        const int pad = ((keys + 15) & ~15) - keys;
                        uint8_t* v = smem + L::kRingOff + stage * L::kTile;
                        for (int i = rloc; i < pad * (D / 8); i += 128) {
                            const int row = keys + i / (D / 8), c8 = i % (D / 8);
                            *reinterpret_cast<uint4*>(v + (c8 >> 3) * (kBc * 128) + row * 128 + (c8 & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
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
                    auto exp_chunk = [&](const float* sc, uint32_t col) {
                        const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
                        uint32_t pk[16];
#pragma unroll
                        for (int c = 0; c < 16; c += 2) {
                            float x0, x1, x2, x3;
                            ffma2(x0, x1, sc[2 * c], sc[2 * c + 1], sl2, -m_use);
                            ffma2(x2, x3, sc[2 * c + 2], sc[2 * c + 3], sl2, -m_use);
                            const float a0 = ex2_approx(x0), b0 = ex2_approx(x1);
                            const float a1 = ex2_approx(x2), b1 = ex2_approx(x3);
                            fadd2(acc0, acc1, a0, b0);
                            fadd2(acc2, acc3, a1, b1);
                            pk[c] = pack_bf16x2(a0, b0);
                            pk[c + 1] = pack_bf16x2(a1, b1);
                        }
                        tmem_st16(t_s + col, pk);
                    };
                    if (key0 + kBc <= all_see) {  // every row sees all 128 keys
                        uint32_t r0[32], r1[32], r2[32], r3[32];
                        tmem_ld32(t_s + 0, r0);
                        tmem_ld32(t_s + 32, r1);
                        tmem_wait_ld(r0);
                        tmem_wait_ld(r1);
                        tmem_ld32(t_s + 64, r2);
                        tmem_ld32(t_s + 96, r3);
                        float* s0 = reinterpret_cast<float*>(r0);
                        float* s1 = reinterpret_cast<float*>(r1);
                        float* s2 = reinterpret_cast<float*>(r2);
                        float* s3 = reinterpret_cast<float*>(r3);
                        float mx0 = fmax3(s0[0], s0[1], s0[2]), mx1 = fmax3(s1[0], s1[1], s1[2]);
#pragma unroll
                        for (int c = 3; c < 31; c += 2) {
                            mx0 = fmax3(mx0, s0[c], s0[c + 1]);
                            mx1 = fmax3(mx1, s1[c], s1[c + 1]);
                        }
                        mx0 = fmax3(mx0, s0[31], fmaxf(mx1, s1[31]));
                        tmem_wait_ld(r2);
                        tmem_wait_ld(r3);
                        float mx2 = fmax3(s2[0], s2[1], s2[2]), mx3 = fmax3(s3[0], s3[1], s3[2]);
#pragma unroll
                        for (int c = 3; c < 31; c += 2) {
                            mx2 = fmax3(mx2, s2[c], s2[c + 1]);
                            mx3 = fmax3(mx3, s3[c], s3[c + 1]);
                        }
                        refer(fmax3(mx0, fmax3(mx2, s2[31], mx3), s3[31]));
                        exp_chunk(s0, 0);
                        exp_chunk(s1, 16);
                        rescale();
                        tmem_wait_st();
                        tc_fence_before_sync();
                        mbar_arrive(bar(L::kPHalf + t));
                        exp_chunk(s2, 32);
                        exp_chunk(s3, 48);
                    } else {
                        // A tail, or later tokens' keys: chunk by chunk in little code, reading the
                        // scores twice.  Chunks past the last key are left out (the output product
                        // stops at the step of 16 that holds it).  P of chunk i overwrites scores of
                        // chunk i / 2, which has been read.
                        const int nch = (keys + 31) >> 5;
                        uint32_t r[32];
                        float* sc = reinterpret_cast<float*>(r);
                        float mx = -INFINITY;
#pragma unroll 1
                        for (int i = 0; i < nch; ++i) {
                            tmem_ld32(t_s + 32 * i, r);
                            tmem_wait_ld(r);
                            const int seen = lim - key0 - 32 * i;  // visible keys from here on
#pragma unroll
                            for (int c = 0; c < 32; ++c) mx = fmaxf(mx, c < seen ? sc[c] : -INFINITY);
                        }
                        refer(mx);
                        rescale();
#pragma unroll 1
                        for (int i = 0; i < nch; ++i) {
                            tmem_ld32(t_s + 32 * i, r);
                            tmem_wait_ld(r);
                            const int seen = lim - key0 - 32 * i;
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (c >= seen) sc[c] = -INFINITY;
                            exp_chunk(sc, 16 * i);
                        }
                        tmem_wait_st();
                        tc_fence_before_sync();
                        mbar_arrive(bar(L::kPHalf + t));
                    }
                    l += (acc0 + acc1) + (acc2 + acc3);
                    tmem_wait_st();
                    tc_fence_before_sync();
                    mbar_arrive(bar(L::kPFull + t));
                }
                if (!ok) break;
                // Epilogue: this piece's O / l (fp32) and log-sum-exp, for the combine kernel.
                ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kOFull + t), (o_phase >> t) & 1u, ctx));
                if (!ok) break;
                const bool merge = both && !two;
                float w_own = 1.f, w_other = 0.f;  // of this chain's O and the other's
                float m = m_ref, sum = l;
                if (merge) {
                    // chain 1's (m, l) through shared memory, then chain 0's through the same place
                    if (t == 1) {
                        xchg[rloc] = make_float2(m_ref, l);
                        mbar_arrive(bar(L::kX + 1));
                    }
                    ok = mbar_wait(bar(L::kX + (t ^ 1)), x_cnt & 1u, ctx) &&
                         mbar_wait(bar(L::kOFull + (t ^ 1)), (o_phase >> (t ^ 1)) & 1u, ctx);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    const float2 other = xchg[rloc];
                    if (t == 0) {
                        xchg[rloc] = make_float2(m_ref, l);
                        mbar_arrive(bar(L::kX + 0));
                    }
                    m = fmaxf(m_ref, other.x);
                    w_own = m_ref == -INFINITY ? 0.f : ex2_approx(m_ref - m);
                    w_other = other.x == -INFINITY ? 0.f : ex2_approx(other.x - m);
                    // a chain whose reference never moved has l = 0, or a NaN to pass on
                    sum = (m_ref == -INFINITY ? l : l * w_own) + (other.x == -INFINITY ? other.y : other.y * w_other);
                }
                tc_fence_after_sync();
                // a row that sees no key of this piece: O = 0, LSE = -inf
                const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
                if (warp_on) {
                    const int64_t part = reinterpret_cast<const volatile PrefixItem*>(
                                             smem + L::kItemOff + (n % kPfxItemRing) * sizeof(PrefixItem))->part + k * p.qrows;
                    const int c0 = merge ? t * (D / 2) : 0, c1 = merge ? c0 + D / 2 : D;
                    const float wa = w_own * inv, wb = w_other * inv;
                    // evict-last: read back right after this grid
                    const uint64_t keep = l2_policy_evict_last();
                    const int here = nrow - quad * 32;  // rows of this warp
                    float* out = p.part_o + (part + quad * 32 + (lane >> 2)) * D + (lane & 3) * 2;
#pragma unroll 1
                    for (int half = 0; half < 32 && half < here; half += 16) {
                        // the weights of this thread's two rows
                        const int ra = half + (lane >> 2);
                        const float wa0 = __shfl_sync(0xffffffffu, wa, ra), wa1 = __shfl_sync(0xffffffffu, wa, ra + 8);
                        const float wb0 = __shfl_sync(0xffffffffu, wb, ra), wb1 = __shfl_sync(0xffffffffu, wb, ra + 8);
                        const uint32_t lanes = static_cast<uint32_t>(half) << 16;
#pragma unroll 1
                        for (int c = c0; c < c1; c += 32) {
                            uint32_t oa[16];
                            tmem_ld16x256(t_o + lanes + t * D + c, oa);
                            if (merge) {
                                uint32_t ob[16];
                                tmem_ld16x256(t_o + lanes + (t ^ 1) * D + c, ob);
                                tmem_wait_ld16(oa);
                                tmem_wait_ld16(ob);
                                // a chain without a visible key for the row has weight 0 and finite O
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    oa[i] = __float_as_uint(__uint_as_float(oa[i]) * ((i & 2) ? wa1 : wa0) +
                                                            __uint_as_float(ob[i]) * ((i & 2) ? wb1 : wb0));
                            } else {
                                tmem_wait_ld16(oa);
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    oa[i] = __float_as_uint(__uint_as_float(oa[i]) * ((i & 2) ? wa1 : wa0));
                            }
                            float* o0 = out + half * D + c;
#pragma unroll
                            for (int i = 0; i < 16; i += 4) {
                                if (ra < here)
                                    st_global_v2_hint(o0 + 2 * i, __uint_as_float(oa[i]), __uint_as_float(oa[i + 1]), keep);
                                if (ra + 8 < here)
                                    st_global_v2_hint(o0 + 8 * D + 2 * i, __uint_as_float(oa[i + 2]),
                                                      __uint_as_float(oa[i + 3]), keep);
                            }
                        }
                    }
                    if (row_on && (!merge || t == 0))
                        st_global_hint(p.part_lse + part + rloc,
                                       sum == 0.f ? -INFINITY : (m + lg2_approx(sum)) * kLn2, keep);
                }
                tc_fence_before_sync();
                if (merge) {
                    mbar_arrive(bar(L::kOEmpty + 0));
                    mbar_arrive(bar(L::kOEmpty + 1));
                    ++x_cnt;
                } else {
                    mbar_arrive_n(bar(L::kOEmpty + t), 2);
                }
            }
            o_phase ^= both ? 3u : 1u << par;
            ring += 2 * nt;
            par = two ? 0u : (par + nt) & 1u;
            __syncwarp();  // every lane has read the ring entry
            if (lane == 0) mbar_arrive(bar(L::kItemEmpty + n % kPfxItemRing));
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
    // The own kernel may still run (this grid does not read what it writes): it has ended when this
    // grid has, so that the combine kernel, which waits for this grid, finds both kernels' pieces.
    if (p.workers > 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---------------------------------------------------------------------------
// Own keys of requests with few rows a key head (the usual decoding step).  A
// piece of one request at one key head and up to 16 rows (whole heads of the group) is bound by
// reading K and V: a warp is enough for it, and many warps with a piece each hide the latency that
// the roles of the kernel above hand from one to the next (2048 pieces of 16 keys: 47 us
// there, 18 us here).  Each warp streams K and V in steps of 16 keys through a ring of its own,
// filled by TMA some steps ahead, across the ends of pieces; Q comes with a
// piece's first step.  S = Q K^T and O += P V as mma.sync m16n8k16 on
// registers: the tensor work is a few percent of a step's time, so the rate of
// these instructions does not matter, and a 128-row tcgen05 tile would be
// seven eighths empty.
// ---------------------------------------------------------------------------
// Eight warps with two steps of 16 keys in flight each (128 KB an SM): 64 pieces of 16384 keys in 91 us
// (5.9 TB/s), 2048 of 256 in 54 us.  A warp's own chain (wait, products, softmax, next copies) is
// about 1 us a step, so warps count and depth does not: seven with three steps 94 and 56 us, six with
// four 101 and 59 us, five with four 121 and 66 us.
constexpr int kOwnWarps = 8;
constexpr int kOwnRows = 16;
// Requests with more rows take several row blocks, whose K/V come from L2 for all but the first.
// That pays up to kOwnMostRows rows (four blocks) on short caches: 64 requests x 8 heads of 20 rows, 64 keys
// 18.5 us (26.8 us as items of the prefix kernel), 600 keys 51 (60) us; on 8 requests of
// 8192 keys it does not: 88 (61) us.
constexpr int kOwnMostRows = 64;
constexpr int kOwnMostKeys = 1024;   // of a cache, for requests of more than one block

template <int D>
struct OwnSmem {
    static constexpr int kPart = kOwnStep * D * 2;         // K or V of a step, or Q of a piece
    static constexpr int kStage = 2 * kPart;
    static constexpr int kStages = D == 128 ? 2 : 4;
    static constexpr int kQSlots = 2;                      // pieces whose Q may be in flight or waiting
    static constexpr int kQOff = kStages * kStage;
    static constexpr int kWarp = kQOff + kQSlots * kPart;
    static constexpr int kStepOff = kOwnWarps * kWarp;     // [warps][stages] OwnStep
    static constexpr int kBarOff = kStepOff + kOwnWarps * kStages * 32;
    static constexpr int kFlagOff = kBarOff + kOwnWarps * kStages * 8;
    static constexpr int kBytes = kFlagOff + 16 + kSmemAlign;
    static_assert(kPart % 1024 == 0, "swizzle atoms");
    static_assert(kBytes <= kSmemLimit, "shared memory");
};
struct OwnStep {
    int req, head, key0, len;
    int rows;             // of its piece, whose
    int edge;             // ... first step this is (bit 0), or last (bit 1)
    int64_t part;         // the piece's partial rows
};
static_assert(sizeof(OwnStep) == 32, "OwnSmem");

// The line of own work as this kernel cuts it: a sequence (request, key head,
// row block) is one unit and then its steps; every worker (warp) has `cap` units.
struct WarpCut {
    int cap;
    __device__ __forceinline__ WarpCut(int total, int workers) {
        cap = (total + workers - 1) / workers;
        if (cap < 1) cap = 1;
    }
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// c[16 x 8] += a[16 x 16] b[16 x 8], bf16 with fp32 accumulation
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
__global__ void __launch_bounds__(kOwnWarps * 32, 1)
attn_prefix_own_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ PrefixParams p) {
    using L = OwnSmem<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int lane = threadIdx.x & 31;
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::kFlagOff);
    const WaitCtx ctx{abort_flag, p.error_word, p.timeout_ns};
    const uint32_t bars = smem_u32(smem) + L::kBarOff + warp * L::kStages * 8;
    const uint32_t ring = smem_u32(smem) + warp * L::kWarp;
    OwnStep* steps = reinterpret_cast<OwnStep*>(smem + L::kStepOff) + warp * L::kStages;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) *abort_flag = 0u;
    if (lane == 0) {
        for (int s = 0; s < L::kStages; ++s) mbar_init(bars + 8 * s, 1);
        fence_barrier_init();
        tma_prefetch_desc(&tmap_q);
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
    }
    __syncthreads();

    // ---- this warp's stretch of the line
    const int worker = blockIdx.x * kOwnWarps + warp;
    const int run = (p.R + 31) / 32;
    int mine = 0;
#pragma unroll 8
    for (int i = 0; i < run; ++i) {
        const int r = lane * run + i;
        mine += warp_seq_cost(r < p.R ? own_len(p, r) : 0);
    }
    const int seqs = p.Hk * p.oblocks;
    mine *= seqs;
    const int upto = warp_scan(mine, lane);
    const int total = __shfl_sync(0xffffffffu, upto, 31);
    const WarpCut cut(total, p.workers);
    const int x0 = static_cast<int>(min(static_cast<int64_t>(worker) * cut.cap, static_cast<int64_t>(total)));
    const int x1 = min(cut.cap, total - x0) + x0;

    // ---- the walk of the issuing side (the same in every lane): request r, its sequence h, steps [s, s1)
    int r = 0, h = 0, s = 0, s1 = 0, s_first = 0, len = 0;
    int window = 0, len_l = 0;       // lens of requests [window, window + 32), one a lane
    int start = 0;                   // of the sequence (r, h)
    bool more = x0 < x1;
    auto len_of = [&](int i) -> int {
        if (i >= window + 32) {
            window = i;
            len_l = window + lane < p.R ? own_len(p, window + lane) : 0;
        }
        return __shfl_sync(0xffffffffu, len_l, i - window);
    };
    // the steps of sequence (r, h) in the stretch; moves on over sequences that have none
    auto settle = [&]() {
        while (more) {
            if (start >= x1 || r >= p.R) {
                more = false;
                break;
            }
            const int cost = warp_seq_cost(len);
            if (len > 0 && start + cost > x0) {
                const int f = start + 1;  // step 0's unit
                s = x0 > f ? x0 - f : 0;
                s1 = min(x1 - f, cost - 1);
                s_first = s;
                if (s < s1) break;
            }
            start += cost;
            if (len == 0 || ++h == seqs) {
                h = 0;
                if (++r < p.R) len = len_of(r);
            }
        }
    };
    if (more) {
        const int at = __ffs(__ballot_sync(0xffffffffu, upto > x0)) - 1;
        r = at * run;
        start = __shfl_sync(0xffffffffu, upto - mine, at);
        window = r - 32;
        len = len_of(r);
        // skip whole requests before the stretch, then whole sequences
        while (r < p.R && start + warp_seq_cost(len) * seqs <= x0) {
            start += warp_seq_cost(len) * seqs;
            if (++r < p.R) len = len_of(r);
        }
        const int cost = warp_seq_cost(len);
        if (cost > 0) {
            h = (x0 - start) / cost;
            start += h * cost;
        }
        settle();
    }
    uint32_t filled = 0, used = 0;
    uint32_t q_filled = 0, q_used = 0;   // pieces whose Q was asked for, and read
    // Asks for the next step while there is a stage for it, and a place for its Q if it begins a piece.
    auto issue = [&]() -> bool {
        if (!more || filled - used == L::kStages || (s == s_first && q_filled - q_used == L::kQSlots)) return false;
        const uint32_t st = filled % L::kStages;
        if (lane == 0) {
            OwnStep d;
            const int blk = h % p.oblocks;
            d.req = r;
            d.head = h / p.oblocks;
            d.key0 = s * kOwnStep;
            d.len = len;
            d.rows = min(p.orows, p.GT - blk * p.orows);
            d.edge = (s == s_first ? 1 : 0) | (s + 1 == s1 ? 2 : 0);
            d.part = p.own_first + (static_cast<int64_t>(r) * seqs + h + worker) * p.orows;
            steps[st] = d;
            const uint32_t full = bars + 8 * st;
            const uint32_t dst = ring + st * L::kStage;
            mbar_arrive_expect_tx(full, 2 * L::kPart + (d.edge & 1 ? p.orows * D * 2 : 0));
#pragma unroll
            for (int b = 0; b < D / 64; ++b) {
                const uint32_t o = dst + b * (kOwnStep * 128);
                if (d.edge & 1)
                    tma_load_5d(ring + L::kQOff + (q_filled % L::kQSlots) * L::kPart + b * (kOwnStep * 128), &tmap_q, full, b * 64,
                                0, blk * p.orows / p.T, d.head, r);
                tma_load_4d(o, &tmap_k, full, b * 64, d.key0, d.head, r);
                tma_load_4d(o + L::kPart, &tmap_v, full, b * 64, d.key0, d.head, r);
            }
        }
        __syncwarp();
        ++filled;
        if (s == s_first) ++q_filled;
        if (++s == s1) {
            start += warp_seq_cost(len);
            if (++h == seqs) {
                h = 0;
                if (++r < p.R) len = len_of(r);
            }
            settle();
        }
        return true;
    };
    while (issue()) {
    }

    // ---- the consuming side
    uint32_t qf[D / 16][4];
    float o[D / 8][4];
    float m[2], l[2];             // rows lane / 4 and lane / 4 + 8
    int hide[2];                  // the last keys these rows do not see
    const int row0 = lane >> 2;
    bool valid[2] = {false, false};   // whether the piece has them
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        hide[i] = p.T - 1 - (row0 + 8 * i) % p.T;  // (a block begins with a head)
        m[i] = -INFINITY;
        l[i] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    const uint32_t lo8 = lane & 7;
    // ldmatrix row addresses: Q and V take rows (lane & 15), K rows (lane & 7) + 8 (lane / 16)
    const uint32_t qv_row = lane & 15, qv_ch = lane >> 4;
    const uint32_t k_row = (lane & 7) + ((lane >> 4) << 3), k_ch = (lane >> 3) & 1;
    const float sign = p.negate_scores ? -1.f : 1.f;
    bool ok = true;
    while (used < filled) {
        const uint32_t st = used % L::kStages;
        ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * st, (used / L::kStages) & 1u, ctx));
        if (!ok) break;
        const uint32_t kb = ring + st * L::kStage, vb = kb + L::kPart;
        const OwnStep d = steps[st];
        if (d.edge & 1) {
            valid[0] = row0 < d.rows;
            valid[1] = row0 + 8 < d.rows;
            const uint32_t qb = ring + L::kQOff + (q_used % L::kQSlots) * L::kPart;
            ++q_used;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t c = 2 * kk + qv_ch;
                ldmatrix4(qb + (c >> 3) * (kOwnStep * 128) + qv_row * 128 + (((c & 7) ^ lo8) << 4), qf[kk]);
            }
        }
        // Cache rows past the last key may hold anything; a zero weight does not undo a NaN in V.
        const int keys = d.len - d.key0;
        if (keys < kOwnStep) {
            for (int i = lane; i < (kOwnStep - keys) * (D / 8); i += 32) {
                const int row = keys + i / (D / 8), c8 = i % (D / 8);
                *reinterpret_cast<uint4*>(smem + (vb - smem_u32(smem)) + (c8 >> 3) * (kOwnStep * 128) + row * 128 +
                                          (c8 & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();  // before the copy that fills this place next
            __syncwarp();
        }
        float sc[2][2][4] = {};  // two chains of products for each of two groups of 8 keys
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t c = 2 * kk + k_ch;
            uint32_t kf[4];
            ldmatrix4(kb + (c >> 3) * (kOwnStep * 128) + k_row * 128 + (((c & 7) ^ lo8) << 4), kf);
            mma_16816(sc[kk & 1][0], qf[kk], kf[0], kf[1]);
            mma_16816(sc[kk & 1][1], qf[kk], kf[2], kf[3]);
        }
        float x[2][4];
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[g][i] = (sc[0][g][i] + sc[1][g][i]) * sign;
        if (keys < kOwnStep + p.T - 1) {
            const int c = d.key0 + (lane & 3) * 2;
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c + 8 * g + (i & 1) >= d.len - hide[i >> 1]) x[g][i] = -INFINITY;
        }
        bool grow = false;
        float alpha[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float mx = fmaxf(fmaxf(x[0][2 * i], x[0][2 * i + 1]), fmaxf(x[1][2 * i], x[1][2 * i + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float m_tile = mx == -INFINITY ? -INFINITY : mx * p.max_scale_log2;
            alpha[i] = 1.f;
            if (valid[i] && m_tile > m[i] + kRescaleLog2Bf16) {
                alpha[i] = ex2_approx(m[i] - m_tile);
                m[i] = m_tile;
                grow = true;
            }
        }
        if (__any_sync(0xffffffffu, grow) && !(d.edge & 1)) {
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                o[j][0] *= alpha[0];
                o[j][1] *= alpha[0];
                o[j][2] *= alpha[1];
                o[j][3] *= alpha[1];
            }
            l[0] *= alpha[0];
            l[1] *= alpha[1];
        }
        uint32_t pf[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float mu = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const float a = ex2_approx(fmaf(x[g][2 * i], p.scale_log2, -mu));
                const float b = ex2_approx(fmaf(x[g][2 * i + 1], p.scale_log2, -mu));
                l[i] += a + b;
                pf[2 * g + i] = pack_bf16x2(a, b);
            }
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            const uint32_t c = 2 * j + qv_ch;
            uint32_t vf[4];
            ldmatrix4_trans(vb + (c >> 3) * (kOwnStep * 128) + qv_row * 128 + (((c & 7) ^ lo8) << 4), vf);
            mma_16816(o[2 * j], pf, vf[0], vf[1]);
            mma_16816(o[2 * j + 1], pf, vf[2], vf[3]);
        }
        __syncwarp();  // every lane has read the step
        ++used;
        while (issue()) {
        }
        if (d.edge & 2) {
            const uint64_t keep = l2_policy_evict_last();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float sum = l[i];
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                // a row that sees no key of this piece: O = 0, LSE = -inf
                const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
                if (valid[i]) {
                    const int64_t row = d.part + row0 + 8 * i;
                    float* dst = p.part_o + row * D + (lane & 3) * 2;
#pragma unroll
                    for (int j = 0; j < D / 8; ++j)
                        st_global_v2_hint(dst + 8 * j, o[j][2 * i] * inv, o[j][2 * i + 1] * inv, keep);
                    if ((lane & 3) == 0)
                        st_global_hint(p.part_lse + row, sum == 0.f ? -INFINITY : (m[i] + lg2_approx(sum)) * kLn2, keep);
                }
                m[i] = -INFINITY;
                l[i] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        }
    }
    // after an abort, the copies in flight land before the shared memory is released
    for (; used < filled; ++used)
        mbar_wait_drain(bars + 8 * (used % L::kStages), (used / L::kStages) & 1u, 50000000ull);
    // One warp leaves every request's start and the total for the combine kernel.
    if (worker == p.workers - 1) {
        int at = 0;
        for (int r0 = 0; r0 < p.R; r0 += 32) {
            const int c = r0 + lane < p.R ? warp_seq_cost(own_len(p, r0 + lane)) * seqs : 0;
            const int sum = warp_scan(c, lane);
            if (r0 + lane < p.R) p.own_start[r0 + lane] = at + sum - c;
            at += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (lane == 0) p.own_start[p.R] = at;
    }
}

// Merge each row's pieces: prefix segments, then own pieces.  WARPS warps per
// row (pieces dealt to them in order, each with a running maximum, then merged
// in a fixed order); lane l holds columns [kPer l, kPer l + kPer).  Requests
// with a negative own length are padding: their rows are left as they were.
template <int D, int WARPS>
__global__ void __launch_bounds__(256) attn_prefix_combine_kernel(const __grid_constant__ PrefixParams p, int grid) {
    constexpr int kPer = D / 32;
    constexpr int kRows = 8 / WARPS;  // rows per CTA
    __shared__ float s_acc[8][D];
    __shared__ float2 s_stat[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int part = warp % WARPS;
    const uint32_t rows = static_cast<uint32_t>(p.R) * p.Hk * p.GT;  // below 2^31
    const uint32_t row = blockIdx.x * kRows + warp / WARPS;          // (r, hq, t)
    const uint32_t hgt = p.Hk * p.GT;
    const int r = row < rows ? static_cast<int>(row / hgt) : 0;
    const int rem = static_cast<int>(row - r * hgt);
    const int h = rem / p.GT, x = rem - h * p.GT;  // key head, row within the request
    const int raw_len = p.lens ? __ldg(p.lens + r) : 0;  // an input: no need to wait for it
    const bool on = row < rows && raw_len >= 0;
    int64_t pstep = 0, pfirst = 0;
    int segs = 0;
    int64_t ofirst = 0;
    auto find_prefix = [&](int own_total) {
        if (!on || p.P == 0) return;
        const PrefixCut cut(p, own_total);
        const int base = p.by_head ? 0 : h * p.ptiles;  // the head's first tile in its run
        const int i0 = cut.run_of(p, base);
        segs = cut.run_of(p, base + p.ptiles - 1) - i0 + 1;
        pfirst = cut.part(p, i0, h) + static_cast<int64_t>(r) * p.GT + x;
        pstep = static_cast<int64_t>(p.R) * p.GT;
    };
    if (p.early == 0) find_prefix(0);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int len = min(raw_len, p.C);
    const int total = p.C > 0 ? __ldcg(p.own_start + p.R) : 0;
    if (p.early > 0) find_prefix(total);
    int pieces = segs;
    if (on && len > 0) {
        int a, b;
        const int q = h * p.oblocks + x / p.orows;
        if (p.workers > 0) {
            const WarpCut cut(total, p.workers);
            const int first = __ldcg(p.own_start + r) + q * warp_seq_cost(len) + 1;
            a = first / cut.cap;
            b = (first + (len - 1) / kOwnStep) / cut.cap;
        } else {
            const OwnCut cut(p, total, grid);
            const int first = __ldcg(p.own_start + r) + q * seq_cost(len) + kPfxItemCost;
            a = cut.cta_of(first);
            b = cut.cta_of(first + (len - 1) / kBc * kPfxTileCost);
        }
        ofirst = p.own_first + (static_cast<int64_t>(r) * p.Hk * p.oblocks + q + a) * p.orows + x % p.orows;
        pieces += b - a + 1;
    }
    auto at = [&](int i) -> int64_t { return i < segs ? pfirst + i * pstep : ofirst + static_cast<int64_t>(i - segs) * p.orows; };
    float acc[kPer];
#pragma unroll
    for (int c = 0; c < kPer; ++c) acc[c] = 0.f;
    float sum = 0.f, mx = -INFINITY;
    constexpr int kUnroll = 6;
    for (int i0 = part; i0 < pieces; i0 += WARPS * kUnroll) {
        float v[kUnroll][kPer], ls[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * WARPS;
            ls[u] = -INFINITY;
#pragma unroll
            for (int c = 0; c < kPer; ++c) v[u][c] = 0.f;
            if (i < pieces) {
                const int64_t idx = at(i);
                ls[u] = __ldcg(p.part_lse + idx);
                CombineVec<D>::load(p.part_o + idx * D + lane * kPer, v[u]);
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
            const float w = ls[u] == -INFINITY ? 0.f : expf(ls[u] - mx);
            sum += w;
#pragma unroll
            for (int c = 0; c < kPer; ++c) acc[c] = fmaf(w, v[u][c], acc[c]);
        }
    }
    if (WARPS > 1) {
#pragma unroll
        for (int c = 0; c < kPer; ++c) s_acc[warp][lane * kPer + c] = acc[c];
        if (lane == 0) s_stat[warp] = make_float2(mx, sum);
        __syncthreads();
        if (part != 0) return;
        float m = mx;
        for (int k = 1; k < WARPS; ++k) m = fmaxf(m, s_stat[warp + k].x);
        const float keep = mx == -INFINITY ? 0.f : expf(mx - m);
        sum = mx == -INFINITY ? sum : sum * keep;  // (a NaN stays)
#pragma unroll
        for (int c = 0; c < kPer; ++c) acc[c] *= keep;
        for (int k = 1; k < WARPS; ++k) {
            const float2 o = s_stat[warp + k];
            const float w = o.x == -INFINITY ? 0.f : expf(o.x - m);
            sum += o.x == -INFINITY ? o.y : o.y * w;
#pragma unroll
            for (int c = 0; c < kPer; ++c) acc[c] = fmaf(w, s_acc[warp + k][lane * kPer + c], acc[c]);
        }
        mx = m;
    }
    if (!on) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no visible key at all: O = 0, LSE = -inf
    const int g = x / p.T, t = x - g * p.T;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + r * p.os[0] + (static_cast<int64_t>(h) * p.G + g) * p.os[1] + t * p.os[2] +
                                                lane * kPer);
#pragma unroll
    for (int c = 0; c < kPer; c += 2) dst[c / 2] = pack_bf16x2(acc[c] * inv, acc[c + 1] * inv);
    if (lane == 0) p.lse[row] = sum == 0.f ? -INFINITY : mx + logf(sum);
}

}  // namespace elsattn
