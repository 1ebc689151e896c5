// Gradients of attention over packed sequences (attn_packed_kernel.cuh), for
// sm_103a, with recomputation as in attn_bwd_kernel.cuh:
//     P = exp(scale * q.k - LSE),  dV = P^T dO,  dP = dO V^T,
//     dS = P * (dP - D), D_i = sum_c dO_ic O_ic,  dQ = scale * dS K,  dK = scale * dS^T Q,
// each query against the keys of its own sequence.  The G query heads of a key
// head are rows (token, head) of one matrix, as in the forward, so that dK and dV
// sum over them in tensor memory.
//
// A unit is a tile of 128 keys of a sequence at one key head; K_j and V_j stay
// in shared memory while blocks of 64 / G tokens (up to 64 rows of Q and dO)
// stream through a TMA ring.  Units lie on a line (LineKeys in packed_line.h)
// that is cut into even stretches, several a CTA so that all CTAs read Q and dO
// of a few heads at a time; a unit that stretches cut leaves its pieces of dK and dV
// in fp32, and attn_packed_bwd_post_kernel adds them up in a fixed order.  dQ
// is summed over the key tiles in fp32 in device memory by bulk reductions, in the order
// in which they come.
//
// The products, their TMEM layout and the warps' shares of them are those of
// attn_bwd_kernel; here the CTA is persistent:
//   warp 0  TMA producer: K_j and V_j of an item, its Q and dO blocks
//   warp 1  tcgen05.mma issuer; owns the TMEM allocation
//   warp 2  row statistics of the blocks into the ring; zeroes rows of other sequences in an item's last block and key tile
//   warp 3  scheduler: the CTA's items, through a ring of descriptions
//   warps 4-7, 12-15  P and dS, then dV;  warps 8-11  dQ readout, then dK
//
// Measured, causal, d = 128: documents of 2000 to 16384 tokens, 16 heads of 8, 3.04 ms, 1.02 PFLOP/s, of which this kernel
// 2.77 (tensor pipe 47 %, shared memory 51 % busy: operands of five products and dS through it); 24 texts of 10 to 2501
// tokens, 24 heads of 4, 741 us, of which this kernel 565 and the two passes over rows 146 (HBM, 6.4 TB/s).  In both this
// kernel is bound by the chain of a block's products: 1.41 us a block and key tile on the documents (1972 an SM), where the products
// alone would take 0.81, and 1.57 on the texts (360 an SM).  Of the texts' blocks 60 of 64 rows are filled (ten tokens of six
// heads), and their tiles cross the diagonal: 16 % more products than the formulas ask for.  The ends of items and the
// imbalance of the CTAs are a tenth of it.
#pragma once

#include <cuda.h>
#include <cstdint>

#include "attn_bwd_kernel.cuh"
#include "attn_packed_kernel.cuh"
#include "packed_line.h"

namespace elsattn {

constexpr int kPkbItemRing = 4;
constexpr int kPkbReaders = 15;  // producer, MMA, statistics, 8 P and dS warps, 4 dQ warps

struct PackedBwdParams {
    const int32_t* q_starts;
    const int32_t* k_starts;
    const float* lse;          // [Hq, Nq]
    const float* dvec;         // [Hq, Nq] -scale * D
    float* dq_acc;             // [Hk, Nq, G, d] fp32, zeroed
    __nv_bfloat16 *dk, *dv;
    int64_t dks[2], dvs[2];    // strides in elements: head, token
    float* part;               // [2 stretches][128 keys][dV | dK][d] fp32, slots as in the forward
    struct PackedBwdCut* cuts; // [stretches]
    int* falls;                // whether q_starts falls somewhere (a sequence's end before its start)
    int R, Hk, G, Nq, Nk;
    int block_tokens, qrows;   // of a query block: whole tokens, and rows
    bool causal;
    int stretches;
    bool whole;                // units are not cut: each is in the stretch that its start is in
    uint32_t* error_word;
    uint64_t timeout_ns;
    float scale, scale_log2;
    uint32_t withhold_first_block;  // test hook: not 0 makes each even CTA arm its first block's barrier without the copies
};

// The unit whose pieces begin in a stretch (pieces: 0 where none is cut there).
struct PackedBwdCut {
    int pieces, head, key0, nkeys;
};

struct PackedBwdItem {
    int nblocks;     // -1: no more items; 0: no token sees the keys
    int head;        // key head
    int tok0;        // first token of the first block, in the tensor
    int ntok;        // tokens from there to the sequence's end
    int key0, nkeys; // the tile's first key in the tensor, and its keys
    int diag;        // the first block's first token sees the tile's keys r <= diag, each next token one more
    int slot;        // partial slot; -1: the unit is whole
};
static_assert(sizeof(PackedBwdItem) == 32, "read by words");

template <int D>
struct PackedBwdLayout {
    static constexpr int kStages = bwd_stages(D);
    static constexpr int kKvTile = 128 * D * 2;
    static constexpr int kQTile = kBq * D * 2;
    static constexpr int kKvBlock = 128 * 128;
    static constexpr int kQBlock = kBq * 128;
    static constexpr int kKOff = 0;
    static constexpr int kVOff = kKvTile;
    static constexpr int kRingOff = 2 * kKvTile;            // stage s: Q_i at +0, dO_i at +kQTile
    static constexpr int kStageBytes = 2 * kQTile;
    static constexpr int kDsOff = kRingOff + kStages * kStageBytes;  // [2][128 keys][64 rows] bf16
    static constexpr int kDsBuf = 128 * kBq * 2;
    static constexpr int kDqOff = kDsOff + 2 * kDsBuf;     // [2 halves][32 rows][d] fp32: dQ_i staged
    static constexpr int kStatOff = kDqOff + kBq * D * 4;  // [stage][lse2 x 64, D x 64] fp32
    static constexpr int kStatBytes = 2 * kBq * 4;
    static constexpr int kItemOff = kStatOff + kStages * kStatBytes;
    static constexpr int kBarOff = kItemOff + kPkbItemRing * static_cast<int>(sizeof(PackedBwdItem));
    static constexpr int kKvFull = 0;                        // K_j and V_j have landed
    static constexpr int kKvZero = 1;                        // rows of a tile that is not full zeroed (such tiles only)
    static constexpr int kQFull = 2;                         // [kStages] Q_i and dO_i have landed
    static constexpr int kQEmpty = kQFull + kStages;         // [kStages]
    static constexpr int kStat = kQEmpty + kStages;          // [kStages] the block's statistics are there, and
                                                             // the rows of a block that is not full zeroed
    static constexpr int kSpFull = kStat + kStages;          // [2] S^T and dP^T of a block complete
    static constexpr int kPFull = kSpFull + 2;               // [2] P^T in TMEM (8 warp arrivals)
    static constexpr int kDsFull = kPFull + 2;               // [2] dS^T in TMEM, dS in shared memory (8)
    static constexpr int kDsEmpty = kDsFull + 2;             // [2] dQ^T MMA done reading dS
    static constexpr int kDqFull = kDsEmpty + 2;             // [2] dQ^T of a block complete
    static constexpr int kDqFree = kDqFull + 2;              // [2] dQ^T read out of TMEM (4)
    static constexpr int kStFull = kDqFree + 2;              // [2] a half of dQ_i staged (4)
    static constexpr int kStEmpty = kStFull + 2;             // [2] the reduction has read that half
    static constexpr int kKvDone = kStEmpty + 2;             // the item's products are complete
    static constexpr int kKvRead = kKvDone + 1;              // dK, dV of an item read out of TMEM (12)
    static constexpr int kDrain = kKvRead + 1;
    static constexpr int kItemFull = kDrain + 1;             // [kPkbItemRing]
    static constexpr int kItemEmpty = kItemFull + kPkbItemRing;
    static constexpr int kNumBars = kItemEmpty + kPkbItemRing;
    static constexpr int kFlagsOff = kBarOff + kNumBars * 8;
    static constexpr int kBytes = kFlagsOff + 16;
    static constexpr int kSmem = kBytes + kSmemAlign;
    static_assert(kSmem <= kSmemLimit, "shared memory");
    static_assert(2 * kSmem > 233472, "one CTA per SM: each allocates all TMEM columns");
    static_assert(kRingOff % 1024 == 0 && kStageBytes % 1024 == 0 && kQTile % 1024 == 0 && kDsOff % 1024 == 0,
                  "swizzle atoms are 1024-byte aligned");
    static_assert(kDqOff % 16 == 0 && kStatOff % 16 == 0 && kItemOff % 16 == 0 && kBarOff % 8 == 0, "alignment");
};

// Element-wise fp32 add of `bytes` (a multiple of 16) of shared memory to global memory, both 16-byte
// aligned; tracked by the issuing thread's bulk groups.
__device__ __forceinline__ void bulk_reduce_add(float* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.reduce.async.bulk.global.shared::cta.bulk_group.add.f32 [%0], [%1], %2;" ::"l"(
                     reinterpret_cast<uint64_t>(dst)),
                 "r"(src), "r"(bytes)
                 : "memory");
}

struct PackedBwdSeq {
    LineKeys line;
    int q0, k0;
};
__device__ __forceinline__ PackedBwdSeq packed_bwd_seq(const PackedBwdParams& p, int r) {
    PackedBwdSeq s;
    auto clip = [](int x, int n) { return min(max(x, 0), n); };
    s.line.block_tokens = p.block_tokens;
    s.line.causal = p.causal;
    s.q0 = clip(__ldg(p.q_starts + r), p.Nq);
    s.k0 = clip(__ldg(p.k_starts + r), p.Nk);
    s.line.nq = max(0, clip(__ldg(p.q_starts + r + 1), p.Nq) - s.q0);
    s.line.nk = max(0, clip(__ldg(p.k_starts + r + 1), p.Nk) - s.k0);
    return s;
}

template <int D>
__global__ void __launch_bounds__(kBwdThreads, 1)
attn_packed_bwd_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_do,
                       const __grid_constant__ PackedBwdParams p) {
    using L = PackedBwdLayout<D>;
    constexpr int kStages = L::kStages;
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
        mbar_init(bar(L::kKvFull), 1);
        mbar_init(bar(L::kKvZero), 1);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bar(L::kQFull + s), 1);
            mbar_init(bar(L::kStat + s), 1);
            mbar_init(bar(L::kQEmpty + s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(L::kSpFull + b), 1);
            mbar_init(bar(L::kPFull + b), 8);
            mbar_init(bar(L::kDsFull + b), 8);
            mbar_init(bar(L::kDsEmpty + b), 1);
            mbar_init(bar(L::kDqFull + b), 1);
            mbar_init(bar(L::kDqFree + b), 4);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(bar(L::kStFull + h), 4);
            mbar_init(bar(L::kStEmpty + h), 1);
        }
        mbar_init(bar(L::kKvDone), 1);
        mbar_init(bar(L::kKvRead), 12);
        mbar_init(bar(L::kDrain), 1);
        for (int s = 0; s < kPkbItemRing; ++s) {
            mbar_init(bar(L::kItemFull + s), 1);
            mbar_init(bar(L::kItemEmpty + s), kPkbReaders);
        }
        fence_barrier_init();
        tma_prefetch_desc(&tmap_q);
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
        tma_prefetch_desc(&tmap_do);
    }
    // Rows that no copy writes (64 is not a multiple of G): zero, since their weight is 0 and 0 times a NaN is not.
    for (int i = threadIdx.x; i < kStages * 2 * (D / 64) * (kBq - p.qrows) * 8; i += kBwdThreads) {
        const int ch = i & 7, row = i / 8 % (kBq - p.qrows) + p.qrows, blk = i / 8 / (kBq - p.qrows);
        *reinterpret_cast<uint4*>(smem + L::kRingOff + blk * L::kQBlock + row * 128 + ch * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    // Up to here nothing is read or written that the grid before may write or read (it zeroes dQ's sums
    // and works out D): the setup overlaps its end.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    auto take_item = [&](uint32_t n, PackedBwdItem& it) -> bool {
        const uint32_t s = n % kPkbItemRing;
        if (!__all_sync(0xffffffffu, mbar_wait(bar(L::kItemFull + s), (n / kPkbItemRing) & 1u, ctx))) return false;
        const int* from = reinterpret_cast<const int*>(smem + L::kItemOff + s * sizeof(PackedBwdItem));
        const int word = from[lane & 7];
        it.nblocks = __shfl_sync(0xffffffffu, word, 0);
        it.head = __shfl_sync(0xffffffffu, word, 1);
        it.tok0 = __shfl_sync(0xffffffffu, word, 2);
        it.ntok = __shfl_sync(0xffffffffu, word, 3);
        it.key0 = __shfl_sync(0xffffffffu, word, 4);
        it.nkeys = __shfl_sync(0xffffffffu, word, 5);
        it.diag = __shfl_sync(0xffffffffu, word, 6);
        it.slot = __shfl_sync(0xffffffffu, word, 7);
        if (lane == 0) mbar_arrive(bar(L::kItemEmpty + s));
        return it.nblocks >= 0;
    };
    // Tokens of the item's block i (1 .. block_tokens).
    auto block_tokens = [&](const PackedBwdItem& it, int i) -> int { return min(p.block_tokens, it.ntok - i * p.block_tokens); };

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        bool ok = true;
        uint32_t cnt = 0, items = 0;   // blocks and items so far
        PackedBwdItem it{};
#pragma unroll 1
        for (uint32_t n = 0; ok && take_item(n, it); ++n) {
            if (it.nblocks == 0) continue;
            // K_j and V_j, once the products of the item before have read theirs
            if (items > 0) ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kKvDone), (items - 1) & 1u, ctx));
            if (!ok) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(bar(L::kKvFull), 2 * L::kKvTile);
#pragma unroll
                for (int b = 0; b < D / 64; ++b) {
                    tma_load_3d(s_base + L::kKOff + b * L::kKvBlock, &tmap_k, bar(L::kKvFull), b * 64, it.key0, it.head);
                    tma_load_3d(s_base + L::kVOff + b * L::kKvBlock, &tmap_v, bar(L::kKvFull), b * 64, it.key0, it.head);
                }
            }
            __syncwarp();
            ++items;
#pragma unroll 1
            for (int i = 0; i < it.nblocks; ++i, ++cnt) {
                const uint32_t s = cnt % kStages;
                ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kQEmpty + s), ((cnt / kStages) & 1u) ^ 1u, ctx));
                if (!ok) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(bar(L::kQFull + s), 2 * p.qrows * D * 2);
                    const uint32_t dst = s_base + L::kRingOff + s * L::kStageBytes;
                    const int tok = it.tok0 + i * p.block_tokens;
                    if (!(p.withhold_first_block && blockIdx.x % 2 == 0 && cnt == 0)) {
#pragma unroll
                        for (int b = 0; b < D / 64; ++b) {
                            tma_load_4d(dst + b * L::kQBlock, &tmap_q, bar(L::kQFull + s), b * 64, 0, it.head, tok);
                            tma_load_4d(dst + L::kQTile + b * L::kQBlock, &tmap_do, bar(L::kQFull + s), b * 64, 0, it.head, tok);
                        }
                    }
                }
                __syncwarp();
            }
        }
        // Every issued copy lands before the CTA ends (bounded waits; also on abort).
        if (items > 0) mbar_wait_drain(bar(L::kKvFull), (items - 1) & 1u, 50000000ull);
#pragma unroll 1
        for (uint32_t c = cnt > kStages ? cnt - kStages : 0; c < cnt; ++c)
            mbar_wait_drain(bar(L::kQFull + c % kStages), (c / kStages) & 1u, 50000000ull);
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (as in attn_bwd_kernel)
        constexpr uint32_t id_s = make_idesc_bf16_f32(128, kBq, false, false);  // S^T, dP^T
        constexpr uint32_t id_acc = make_idesc_bf16_f32(128, D, false, true);   // dV, dK (A in TMEM)
        constexpr uint32_t id_dq = make_idesc_bf16_f32(128, kBq, true, true);   // dQ^T (A, B MN-major)
        const uint32_t t_dv = tmem, t_dk = tmem + D;
        const uint64_t dk_k = make_smem_desc_sw128(s_base + L::kKOff, 16, 1024);            // K_j, K-major
        const uint64_t dv_k = make_smem_desc_sw128(s_base + L::kVOff, 16, 1024);            // V_j, K-major
        // K_j^T as A of dQ^T: d-blocks of 64 are L::kKvBlock apart.  For d = 64 the
        // second block (rows 64..127 of dQ^T) reads V_j: those lanes are never used.
        const uint64_t dkt_mn = make_smem_desc_sw128(s_base + L::kKOff, L::kKvBlock, 1024);
        auto kstep_a = [](int kk) { return static_cast<uint64_t>(((kk >> 2) * L::kKvBlock + (kk & 3) * 32) >> 4); };
        auto kstep_b = [](int kk) { return static_cast<uint64_t>(((kk >> 2) * L::kQBlock + (kk & 3) * 32) >> 4); };
        constexpr uint64_t kRows16 = (16 * 128) >> 4;  // 16 rows of an MN-major operand
        auto a_col = [](int kk) { return static_cast<uint32_t>((kk >> 1) * 32 + (kk & 1) * 8); };
        bool ok = true;
        uint32_t cnt = 0, items = 0, tails = 0;
        PackedBwdItem it{};
        // S^T and dP^T of the item's block i, the CTA's block c = cnt + i.  The S^T half is free: P^T of
        // block c - 2 was read by dV (issued earlier) and by the dS pass (its DsFull was awaited).  The
        // dP^T half holds dQ^T of block c - 2 until the readout warps release it.
        auto issue_sdp = [&](int i) -> bool {
            const uint32_t c = cnt + i, s = c % kStages, b = c & 1u;
            const uint32_t q = s_base + L::kRingOff + s * L::kStageBytes;
            bool w = mbar_wait(bar(L::kQFull + s), (c / kStages) & 1u, ctx);
            if (block_tokens(it, i) < p.block_tokens) w = w && mbar_wait(bar(L::kStat + s), (c / kStages) & 1u, ctx);
            if (!__all_sync(0xffffffffu, w)) return false;
            tc_fence_after_sync();
            const uint32_t t_s = tmem + 2 * D + 128 * b;
            const uint64_t dq_k = make_smem_desc_sw128(q, 16, 1024);
            const uint64_t ddo_k = make_smem_desc_sw128(q + L::kQTile, 16, 1024);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) mma_ss(t_s, dk_k + kstep_a(kk), dq_k + kstep_b(kk), id_s, kk > 0 ? 1u : 0u);
            }
            __syncwarp();
            if (c >= 2) {
                w = mbar_wait(bar(L::kDqFree + b), ((c - 2) >> 1) & 1u, ctx);
                if (!__all_sync(0xffffffffu, w)) return false;
                tc_fence_after_sync();
            }
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss(t_s + 64, dv_k + kstep_a(kk), ddo_k + kstep_b(kk), id_s, kk > 0 ? 1u : 0u);
                mma_commit(bar(L::kSpFull + b));
            }
            __syncwarp();
            return true;
        };
#pragma unroll 1
        for (uint32_t n = 0; ok && take_item(n, it); ++n) {
            const int nb = it.nblocks;
            if (nb == 0) continue;
            bool w = mbar_wait(bar(L::kKvFull), items & 1u, ctx);
            if (it.nkeys < kBc) w = w && mbar_wait(bar(L::kKvZero), tails++ & 1u, ctx);
            if (!(ok = __all_sync(0xffffffffu, w))) break;
            ok = issue_sdp(0);
            if (ok && nb > 1) ok = issue_sdp(1);
#pragma unroll 1
            for (int i = 0; i < nb && ok; ++i) {
                const uint32_t c = cnt + i, s = c % kStages, b = c & 1u, ph = (c >> 1) & 1u;
                const uint32_t q = s_base + L::kRingOff + s * L::kStageBytes;
                const uint32_t t_s = tmem + 2 * D + 128 * b;
                const uint64_t dq_mn = make_smem_desc_sw128(q, L::kQBlock, 1024);               // Q_i, MN-major
                const uint64_t ddo_mn = make_smem_desc_sw128(q + L::kQTile, L::kQBlock, 1024);  // dO_i, MN-major
                const uint64_t dds_mn = make_smem_desc_sw128(s_base + L::kDsOff + b * L::kDsBuf, L::kDsBuf, 1024);
                // dV += P^T dO_i once P^T is in TMEM (an item's first one: once dV and dK of the item before are read)
                w = mbar_wait(bar(L::kPFull + b), ph, ctx);
                if (i == 0 && items > 0) w = w && mbar_wait(bar(L::kKvRead), (items - 1) & 1u, ctx);
                if (!(ok = __all_sync(0xffffffffu, w))) break;
                tc_fence_after_sync();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kBq / 16; ++kk)
                        mma_ts(t_dv, t_s + a_col(kk), ddo_mn + kk * kRows16, id_acc, (i > 0 || kk > 0) ? 1u : 0u);
                }
                __syncwarp();
                // dK += dS^T Q_i and dQ_i^T = K_j^T dS^T once dS is ready
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kDsFull + b), ph, ctx)))) break;
                tc_fence_after_sync();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kBq / 16; ++kk)
                        mma_ts(t_dk, t_s + 64 + a_col(kk), dq_mn + kk * kRows16, id_acc, (i > 0 || kk > 0) ? 1u : 0u);
#pragma unroll
                    for (int kk = 0; kk < kBc / 16; ++kk)
                        mma_ss(t_s + 64, dkt_mn + kk * kRows16, dds_mn + kk * kRows16, id_dq, kk > 0 ? 1u : 0u);
                    mma_commit(bar(L::kDqFull + b));
                    mma_commit(bar(L::kDsEmpty + b));
                    mma_commit(bar(L::kQEmpty + s));
                    if (i == nb - 1) mma_commit(bar(L::kKvDone));
                }
                __syncwarp();
                if (i + 2 < nb) ok = issue_sdp(i + 2);
            }
            cnt += nb;
            ++items;
        }
        if (elect_one()) mma_commit(bar(L::kDrain));
        __syncwarp();
        mbar_wait_drain(bar(L::kDrain), 0, 1000000000ull);
    } else if (warp == 2) {
        // ------------------------------------------------------------ row statistics
        // Column c of a block is row c of its tokens' heads: -LSE * log2(e), so that P = 2^(s * scale * log2 e + it),
        // and -scale * D.  Rows that are not there, and rows that see no key, get -inf and 0: P = 0, dS = 0.
        bool ok = true;
        uint32_t cnt = 0, items = 0;
        PackedBwdItem it{};
        const int c0 = lane, c1 = lane + 32;
        const int t0 = c0 / p.G, g0 = c0 - t0 * p.G, t1 = c1 / p.G, g1 = c1 - t1 * p.G;
        auto zero_rows = [&](uint32_t off, int blocks, int block_bytes, int from, int to) {
#pragma unroll 1
            for (int i = lane; i < blocks * (to - from) * 8; i += 32) {
                const int ch = i & 7, row = i / 8 % (to - from) + from, blk = i / 8 / (to - from);
                *reinterpret_cast<uint4*>(smem + off + blk * block_bytes + row * 128 + ch * 16) = make_uint4(0, 0, 0, 0);
            }
        };
#pragma unroll 1
        for (uint32_t n = 0; ok && take_item(n, it); ++n) {
            if (it.nblocks == 0) continue;
            // (waited for at every item: a parity tells one fill from the next, not from the one after)
            ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kKvFull), items & 1u, ctx));
            if (!ok) break;
            if (it.nkeys < kBc) {  // the tile's other rows are another sequence's keys
                zero_rows(L::kKOff, 2 * (D / 64), L::kKvBlock, it.nkeys, kBc);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::kKvZero));
            }
            ++items;
            float l[2], dd[2];  // of the next block
            auto fetch = [&](int i) {
                const int tokens = block_tokens(it, i), tok = it.tok0 + i * p.block_tokens;
                const int64_t h = static_cast<int64_t>(it.head) * p.G;
                const bool on0 = c0 < p.qrows && t0 < tokens, on1 = c1 < p.qrows && t1 < tokens;
                const int64_t a0 = (h + g0) * p.Nq + tok + t0, a1 = (h + g1) * p.Nq + tok + t1;
                l[0] = on0 ? __ldg(p.lse + a0) : -INFINITY;
                l[1] = on1 ? __ldg(p.lse + a1) : -INFINITY;
                dd[0] = on0 ? __ldg(p.dvec + a0) : 0.f;
                dd[1] = on1 ? __ldg(p.dvec + a1) : 0.f;
            };
            fetch(0);
#pragma unroll 1
            for (int i = 0; i < it.nblocks; ++i, ++cnt) {
                const uint32_t s = cnt % kStages;
                float nl[2], nd[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    nl[u] = l[u] == -INFINITY ? -INFINITY : -(l[u] * 1.4426950408889634f);
                    nd[u] = dd[u];
                }
                if (i + 1 < it.nblocks) fetch(i + 1);
                ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kQEmpty + s), ((cnt / kStages) & 1u) ^ 1u, ctx));
                if (!ok) break;
                float* stat = reinterpret_cast<float*>(smem + L::kStatOff + s * L::kStatBytes);
                stat[c0] = nl[0];
                stat[c1] = nl[1];
                stat[kBq + c0] = nd[0];
                stat[kBq + c1] = nd[1];
                const int tokens = block_tokens(it, i);
                if (tokens < p.block_tokens) {  // the block's other rows are another sequence's
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kQFull + s), (cnt / kStages) & 1u, ctx));
                    if (!ok) break;
                    zero_rows(L::kRingOff + s * L::kStageBytes, 2 * (D / 64), L::kQBlock, tokens * p.G, p.qrows);
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::kStat + s));
            }
        }
    } else if (warp == 3) {
        // ------------------------------------------------------------ scheduler
        uint32_t n = 0;
        bool ok = true;
        auto publish = [&](const PackedBwdItem& it) {
            const uint32_t s = n % kPkbItemRing;
            if (n >= kPkbItemRing)  // for a whole item, whose length is the sequence's
                ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kItemEmpty + s), ((n / kPkbItemRing) - 1) & 1u,
                                                       WaitCtx{ctx.abort_flag, ctx.error_word, 16 * ctx.timeout_ns}));
            if (!ok) return;
            if (lane == 0) {
                *reinterpret_cast<PackedBwdItem*>(smem + L::kItemOff + s * sizeof(PackedBwdItem)) = it;
                mbar_arrive(bar(L::kItemFull + s));
            }
            __syncwarp();
            ++n;
        };
        PackedBwdItem it{};
        const int run = (p.R + 31) / 32;
        int64_t mine = 0;
        PackedBwdSeq own{};
        int64_t own_len = 0;
        bool falls = false;
#pragma unroll 1
        for (int i = 0; i < run; ++i) {
            const int r = lane * run + i;
            if (r < p.R) {
                own = packed_bwd_seq(p, r);
                falls = falls || __ldg(p.q_starts + r + 1) < __ldg(p.q_starts + r);
                own_len = own.line.length();
                mine += own_len;
            }
        }
        falls = __any_sync(0xffffffffu, falls);
        if (blockIdx.x == 0 && lane == 0) *p.falls = falls;
        mine *= p.Hk;
        const int64_t upto = warp_scan64(mine, lane);
        const int64_t total = __shfl_sync(0xffffffffu, upto, 31);
        const int64_t len = line_stretch(total, p.stretches, kKeyLineLeast * p.block_tokens);
        // (after a timeout too: what the merging kernel reads of the cuts has to be theirs)
#pragma unroll 1
        for (int i = blockIdx.x; i < p.stretches; i += gridDim.x) {
            const int64_t x0 = i * len;
            const int64_t x1 = min(x0 + len, total);
            PackedBwdCut cut{};
            if (ok && x0 < x1) {
                const int at = run == 1 ? 0 : __ffs(__ballot_sync(0xffffffffu, upto > x0)) - 1;
                int64_t start = __shfl_sync(0xffffffffu, upto - mine, at);
#pragma unroll 1
                for (int r0 = at * run; r0 < p.R && start < x1 && ok; r0 += 32) {
                    if (run > 1) {
                        own_len = 0;
                        if (r0 + lane < p.R) {
                            own = packed_bwd_seq(p, r0 + lane);
                            own_len = own.line.length();
                        }
                    }
                    const int64_t cost = own_len * p.Hk;
                    const int64_t end_l = start + warp_scan64(cost, lane);
                    uint32_t in = __ballot_sync(0xffffffffu, cost > 0 && end_l > x0 && end_l - cost < x1);
#pragma unroll 1
                    for (; in != 0 && ok; in &= in - 1) {
                        const int src = __ffs(in) - 1;
                        PackedBwdSeq s;
                        s.line.nq = __shfl_sync(0xffffffffu, own.line.nq, src);
                        s.line.nk = __shfl_sync(0xffffffffu, own.line.nk, src);
                        s.line.block_tokens = p.block_tokens;
                        s.line.causal = p.causal;
                        s.q0 = __shfl_sync(0xffffffffu, own.q0, src);
                        s.k0 = __shfl_sync(0xffffffffu, own.k0, src);
                        const int64_t first = __shfl_sync(0xffffffffu, end_l - cost, src);
                        const int64_t per = __shfl_sync(0xffffffffu, own_len, src);
                        const int tiles = s.line.tiles();
                        int h = x0 > first ? static_cast<int>(line_div(x0 - first, per)) : 0;
#pragma unroll 1
                        for (int64_t hs = first + h * per; h < p.Hk && hs < x1 && ok; ++h, hs += per) {
                            // the key tile that x0 is in: the last one that begins at or before it
                            int j = 0;
                            if (x0 > hs) {
                                int lo = 0, hi = tiles;  // before(lo) <= x0 - hs, and not before(hi)
                                while (hi - lo > 1) {
                                    const int width = (hi - lo + 31) / 32;
                                    const int probe = lo + lane * width;
                                    const bool below = probe < hi && s.line.before(probe) <= x0 - hs;
                                    const int k = 31 - __clz(__ballot_sync(0xffffffffu, below));  // lane 0 is
                                    lo += k * width;
                                    hi = min(hi, lo + width);
                                }
                                j = lo;
                            }
                            int64_t us = hs + s.line.before(j);
#pragma unroll 1
                            for (; j < tiles && us < x1 && ok; ++j) {
                                const int tok = s.line.first(j), ntok = s.line.nq - tok;
                                const int nb = (ntok + p.block_tokens - 1) / p.block_tokens;
                                const int64_t begin = us + s.line.unit_cost();
                                LinePart part(begin, nb, p.block_tokens, x0, x1);
                                if (p.whole) {
                                    part.t0 = us >= x0 ? 0 : nb;
                                    part.t1 = nb;
                                }
                                if (part.t0 < part.t1 || (nb == 0 && us >= x0)) {
                                    const int skip = nb == 0 ? 0 : part.t0 * p.block_tokens;
                                    it.nblocks = nb == 0 ? 0 : part.t1 - part.t0;
                                    it.head = h;
                                    it.tok0 = s.q0 + tok + skip;
                                    it.ntok = ntok - skip;
                                    it.key0 = s.k0 + j * kLineTile;
                                    it.nkeys = min(kLineTile, s.line.nk - j * kLineTile);
                                    it.diag = p.causal ? (tok + skip - s.line.nq) + (s.line.nk - j * kLineTile) : kLineTile;
                                    it.slot = -1;
                                    if (nb > 0 && it.nblocks < nb) {
                                        it.slot = part.t0 == 0 ? 2 * i + 1 : 2 * i;
                                        if (part.t0 == 0) {
                                            const int64_t last = begin + static_cast<int64_t>(nb - 1) * p.block_tokens;
                                            cut.pieces = static_cast<int>(line_div(last, len)) - i + 1;
                                            cut.head = h;
                                            cut.key0 = it.key0;
                                            cut.nkeys = it.nkeys;
                                        }
                                    }
                                    publish(it);
                                }
                                us += s.line.cost(j);
                            }
                        }
                    }
                    start = __shfl_sync(0xffffffffu, end_l, 31);
                }
            }
            if (lane == 0 && !p.whole) p.cuts[i] = cut;
        }
        it.nblocks = -1;
        if (ok) publish(it);
    } else {
        const bool dq_warp = warp >= 8 && warp < 12;
        const int quad = warp & 3;
        const int r = quad * 32 + lane;       // key row of the tile; in the dQ readout, head-dim column
        const int c0 = warp >= 12 ? 32 : 0;   // P and dS: this warpgroup's columns (rows of the block)
        const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
        bool ok = true;
        uint32_t cnt = 0, items = 0;
        PackedBwdItem it{};
        // columns [from, to) of dV or dK (in TMEM at `col`) of this thread's key row -> bf16, or this piece's in fp32
        auto write_rows = [&](uint32_t col, __nv_bfloat16* dst, const int64_t (&st)[2], int which, int from, int to) {
            const bool key_ok = r < it.nkeys;
            uint4* row = reinterpret_cast<uint4*>(dst + it.head * st[0] + static_cast<int64_t>(it.key0 + (key_ok ? r : 0)) * st[1]);
            if (it.nblocks == 0) {
                if (key_ok)
#pragma unroll 1
                    for (int c = from; c < to; c += 8) row[c / 8] = make_uint4(0, 0, 0, 0);
                return;
            }
            float4* part = reinterpret_cast<float4*>(p.part + ((static_cast<int64_t>(it.slot) * kBc + r) * 2 + which) * D);
#pragma unroll 1
            for (int c = from; c < to; c += 32) {
                uint32_t v[32];
                tmem_ld32(tmem + lane_addr + col + c, v);
                tmem_wait_ld(v);
                if (key_ok && it.slot < 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        row[c / 8 + i] = make_uint4(pack_bf16x2(__uint_as_float(v[8 * i]), __uint_as_float(v[8 * i + 1])),
                                                    pack_bf16x2(__uint_as_float(v[8 * i + 2]), __uint_as_float(v[8 * i + 3])),
                                                    pack_bf16x2(__uint_as_float(v[8 * i + 4]), __uint_as_float(v[8 * i + 5])),
                                                    pack_bf16x2(__uint_as_float(v[8 * i + 6]), __uint_as_float(v[8 * i + 7])));
                } else if (key_ok) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        part[c / 4 + i] = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                                      __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
                }
                __syncwarp();
            }
        };
        auto item_end = [&]() {  // this warp has read its part of dV and dK
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::kKvRead));
            ++items;
        };
        if (!dq_warp) {
            // (x0, x1) = (a0 * b + c0, a1 * b + c1) and (x0, x1) *= (m0, m1) on packed fp32 pairs
            auto ffma2c = [](float& x0, float& x1, float a0, float a1, float b, float c0, float c1) {
                uint64_t rr;
                asm("{\n\t.reg .b64 pa, pb, pc;\n\tmov.b64 pa, {%1, %2};\n\tmov.b64 pb, {%3, %3};\n\t"
                    "mov.b64 pc, {%4, %5};\n\tfma.rn.f32x2 %0, pa, pb, pc;\n\t}"
                    : "=l"(rr) : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
                asm("mov.b64 {%0, %1}, %2;" : "=f"(x0), "=f"(x1) : "l"(rr));
            };
            auto fmul2 = [](float& x0, float& x1, float m0, float m1) {
                uint64_t rr;
                asm("{\n\t.reg .b64 pa, pb;\n\tmov.b64 pa, {%1, %2};\n\tmov.b64 pb, {%3, %4};\n\tmul.rn.f32x2 %0, pa, pb;\n\t}"
                    : "=l"(rr) : "f"(x0), "f"(x1), "f"(m0), "f"(m1));
                asm("mov.b64 {%0, %1}, %2;" : "=f"(x0), "=f"(x1) : "l"(rr));
            };
            // ------------------------------------------------------------ P and dS
            // Thread r = key row r of the tile (TMEM lane r).  Warps 4-7 take the block's rows 0-31,
            // warps 12-15 rows 32-63.
            const float sl2 = p.scale_log2;
#pragma unroll 1
            for (uint32_t n = 0; ok && take_item(n, it); ++n) {
#pragma unroll 1
                for (int i = 0; i < it.nblocks && ok; ++i, ++cnt) {
                    const uint32_t b = cnt & 1u, ph = (cnt >> 1) & 1u, s = cnt % kStages;
                    const uint32_t t_s = tmem + lane_addr + 2 * D + 128 * b, t_dp = t_s + 64;
                    const float* lse2 = reinterpret_cast<const float*>(smem + L::kStatOff + s * L::kStatBytes);
                    const float* dvec = lse2 + kBq;
                    // P in fp32: dS is rounded once (from P rounded to bf16, dQ and dK were off by 1.3 times as much)
                    float pr[32];
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kSpFull + b), ph, ctx) &&
                                                     mbar_wait(bar(L::kStat + s), (cnt / kStages) & 1u, ctx));
                    if (!ok) break;
                    tc_fence_after_sync();
                    {
                        uint32_t sv[32];
                        tmem_ld32(t_s + c0, sv);
                        float l[32];
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            const float4 t = *reinterpret_cast<const float4*>(lse2 + c0 + c);
                            l[c] = t.x, l[c + 1] = t.y, l[c + 2] = t.z, l[c + 3] = t.w;
                        }
                        tmem_wait_ld(sv);
                        uint32_t pk[16];
                        // Key r is seen by the tokens t with r <= diag + t: the columns from `from` on.
                        const int from = r < it.nkeys ? max(0, r - it.diag - i * p.block_tokens) * p.G : kBq;
                        if (__any_sync(0xffffffffu, from > c0)) {
#pragma unroll
                            for (int c = 0; c < 32; c += 2) {
                                float a, bb;
                                ffma2c(a, bb, __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]), sl2, l[c], l[c + 1]);
                                a = ex2_approx(a);
                                bb = ex2_approx(bb);
                                if (c0 + c < from) a = 0.f;
                                if (c0 + c + 1 < from) bb = 0.f;
                                pr[c] = a;
                                pr[c + 1] = bb;
                                pk[c / 2] = pack_bf16x2(a, bb);
                            }
                        } else {
#pragma unroll
                            for (int c = 0; c < 32; c += 2) {
                                float a, bb;
                                ffma2c(a, bb, __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]), sl2, l[c], l[c + 1]);
                                pr[c] = ex2_approx(a);
                                pr[c + 1] = ex2_approx(bb);
                                pk[c / 2] = pack_bf16x2(pr[c], pr[c + 1]);
                            }
                        }
                        tmem_st16(t_s + c0, pk);  // over this warpgroup's own S^T columns
                    }
                    tmem_wait_st();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(L::kPFull + b));
                    __syncwarp();
                    // dS = scale * P * (dP - D): dS^T -> TMEM over dP^T's columns, dS -> shared memory
                    // ([key][row], 128-byte swizzled) for dQ^T.
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kDsEmpty + b), ph ^ 1u, ctx));
                    if (!ok) break;
                    tc_fence_after_sync();
                    uint8_t* ds_row = smem + L::kDsOff + b * L::kDsBuf + r * 128;
                    {
                        uint32_t dv[32];
                        tmem_ld32(t_dp + c0, dv);
                        tmem_wait_ld(dv);
                        uint32_t pk[16];
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            const float4 dd = *reinterpret_cast<const float4*>(dvec + c0 + c);
                            float a, bb;  // scale * dP - scale * D, then times P
                            ffma2c(a, bb, __uint_as_float(dv[c]), __uint_as_float(dv[c + 1]), p.scale, dd.x, dd.y);
                            fmul2(a, bb, pr[c], pr[c + 1]);
                            pk[c / 2] = pack_bf16x2(a, bb);
                            ffma2c(a, bb, __uint_as_float(dv[c + 2]), __uint_as_float(dv[c + 3]), p.scale, dd.z, dd.w);
                            fmul2(a, bb, pr[c + 2], pr[c + 3]);
                            pk[c / 2 + 1] = pack_bf16x2(a, bb);
                        }
                        tmem_st16(t_dp + c0, pk);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int ch = (c0 >> 3) + q;  // 16-byte chunk of the 128-byte row
                            *reinterpret_cast<uint4*>(ds_row + ((ch ^ (r & 7)) << 4)) =
                                make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
                        }
                    }
                    fence_proxy_async_smem();  // dS written by threads, read by the tensor core
                    tmem_wait_st();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(L::kDsFull + b));
                    __syncwarp();
                }
                if (!ok) break;
                // dV of this key tile, half of its columns per warpgroup
                if (it.nblocks > 0) {
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kKvDone), items & 1u, ctx));
                    if (!ok) break;
                    tc_fence_after_sync();
                }
                write_rows(0, p.dv, p.dvs, 0, c0 ? D / 2 : 0, c0 ? D : D / 2);
                if (it.nblocks > 0) item_end();
            }
        } else {
            // ------------------------------------------------------------ dQ readout
            // Thread r = head-dim column r of dQ_i^T (TMEM lane r).  The block's dQ_i is staged in
            // shared memory as two halves of [32 rows][d] fp32, and each half is added to the sums by one
            // bulk reduction while the other half is staged: the block's rows are neighbours there.  One thread
            // issues the reductions; it releases a half once the one issued before the current one has read its data.
            const bool col_ok = r < D;  // warp-uniform: d is a multiple of 32
            const bool issuer = warp == 8 && lane == 0;
            constexpr int kHalf = kBq / 2;
#pragma unroll 1
            for (uint32_t n = 0; ok && take_item(n, it); ++n) {
#pragma unroll 1
                for (int i = 0; i < it.nblocks && ok; ++i, ++cnt) {
                    const uint32_t b = cnt & 1u, ph = (cnt >> 1) & 1u;
                    const uint32_t t_dq = tmem + lane_addr + 2 * D + 128 * b + 64;
                    const int rows = block_tokens(it, i) * p.G;  // of the block
                    float* acc = p.dq_acc + (static_cast<int64_t>(it.head) * p.Nq + it.tok0 + i * p.block_tokens) * p.G * D;
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kDqFull + b), ph, ctx));
                    if (!ok) break;
                    tc_fence_after_sync();
                    uint32_t v[2][32];
                    tmem_ld32(t_dq, v[0]);
                    tmem_ld32(t_dq + 32, v[1]);
                    tmem_wait_ld(v[0]);
                    tmem_wait_ld(v[1]);
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(L::kDqFree + b));
                    __syncwarp();
#pragma unroll
                    for (int h = 0; h < 2 && ok; ++h) {
                        ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kStEmpty + h), (cnt & 1u) ^ 1u, ctx));
                        if (!ok) break;
                        float* stage = reinterpret_cast<float*>(smem + L::kDqOff + h * kHalf * D * 4);
                        if (col_ok) {
#pragma unroll
                            for (int c = 0; c < kHalf; ++c) stage[c * D + r] = __uint_as_float(v[h][c]);
                        }
                        fence_proxy_async_smem();  // staged by threads, read by the bulk copy
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(L::kStFull + h));
                        bool w = true;
                        if (issuer) {
                            w = mbar_wait(bar(L::kStFull + h), cnt & 1u, ctx);
                            const int here = min(kHalf, rows - h * kHalf);
                            if (w && here > 0)
                                bulk_reduce_add(acc + h * kHalf * D, s_base + L::kDqOff + h * kHalf * D * 4, here * D * 4);
                            bulk_commit_group();
                            // the reduction issued before this one has read its half: release it
                            bulk_wait_group_read<1>();
                            if (h == 1) mbar_arrive(bar(L::kStEmpty + 0));
                            else if (cnt > 0) mbar_arrive(bar(L::kStEmpty + 1));
                        }
                        ok = __all_sync(0xffffffffu, w);
                    }
                }
                if (!ok) break;
                // dK of this key tile
                if (it.nblocks > 0) {
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kKvDone), items & 1u, ctx));
                    if (!ok) break;
                    tc_fence_after_sync();
                }
                write_rows(D, p.dk, p.dks, 1, 0, D);
                if (it.nblocks > 0) item_end();
            }
            if (issuer) bulk_wait_group<0>();  // every reduction has landed before the CTA ends
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

struct PackedRowParams {
    const __nv_bfloat16 *o, *dout;
    __nv_bfloat16* dq;
    int64_t os[2], dos[2], dqs[2];  // strides in elements: head, token
    int Hq, G, Nq;
};

// D = sum_c dO_c O_c of every row, stored as dvec = -scale * D, and dQ's sums zeroed.  D / 8 threads a row.
template <int D>
__global__ void __launch_bounds__(256) attn_packed_bwd_prep_kernel(const PackedRowParams q, float* dvec, float* dq_acc, float scale) {
    constexpr int kTpr = D / 8;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the main kernel sets up beside this grid, and waits for it
    const int64_t tid = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int64_t row = tid / kTpr;  // token-major: (token, head)
    const int part = static_cast<int>(tid % kTpr);
    const bool live = row < static_cast<int64_t>(q.Hq) * q.Nq;
    const int tok = live ? static_cast<int>(row / q.Hq) : 0, h = live ? static_cast<int>(row - static_cast<int64_t>(tok) * q.Hq) : 0;
    float acc = 0.f;
    if (live) {
        const uint4 o = __ldg(reinterpret_cast<const uint4*>(q.o + h * q.os[0] + tok * q.os[1]) + part);
        const uint4 g = __ldg(reinterpret_cast<const uint4*>(q.dout + h * q.dos[0] + tok * q.dos[1]) + part);
        const uint32_t ow[4] = {o.x, o.y, o.z, o.w}, gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            acc = fmaf(__uint_as_float(ow[k] << 16), __uint_as_float(gw[k] << 16), acc);
            acc = fmaf(__uint_as_float(ow[k] & 0xffff0000u), __uint_as_float(gw[k] & 0xffff0000u), acc);
        }
        const int hk = h / q.G;
        float4* z = reinterpret_cast<float4*>(dq_acc + ((static_cast<int64_t>(hk) * q.Nq + tok) * q.G + (h - hk * q.G)) * D);
        z[2 * part] = make_float4(0.f, 0.f, 0.f, 0.f);
        z[2 * part + 1] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int off = kTpr / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if (live && part == 0) dvec[static_cast<int64_t>(h) * q.Nq + tok] = -scale * acc;
}

// The first kPkbCutCtas CTAs for each stretch add up the pieces of dK and dV of the unit that begins to be cut there, in the
// pieces' order; the others round dQ's sums to bf16, rows of tokens that are in no sequence left as they were.
constexpr int kPkbCutCtas = 8;   // each has 16 of the tile's 128 keys

template <int D>
__global__ void __launch_bounds__(256, 6) attn_packed_bwd_post_kernel(const __grid_constant__ PackedBwdParams p, const PackedRowParams q) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int kVecs = D / 8;  // 8 elements a thread
    const unsigned cut_ctas = p.whole ? 0u : static_cast<unsigned>(p.stretches) * kPkbCutCtas;
    if (blockIdx.x < cut_ctas) {
        const int i = blockIdx.x / kPkbCutCtas;
        const int* desc = reinterpret_cast<const int*>(p.cuts + i);
        const int pieces = __ldcg(desc);
        if (pieces == 0) return;
        const int head = __ldcg(desc + 1), key0 = __ldcg(desc + 2), nkeys = __ldcg(desc + 3);
        constexpr int kKeys = kBc / kPkbCutCtas;
        const int r0 = (blockIdx.x % kPkbCutCtas) * kKeys;
#pragma unroll
        for (int x = threadIdx.x; x < kKeys * 2 * kVecs; x += 256) {
            const int r = r0 + x / (2 * kVecs), which = x / kVecs & 1, c = x % kVecs * 8;
            if (r >= nkeys) break;
            float acc[8] = {};
            for (int s = 0; s < pieces; ++s) {
                const int64_t slot = s == 0 ? 2 * static_cast<int64_t>(i) + 1 : 2 * (static_cast<int64_t>(i) + s);
                const float4* from = reinterpret_cast<const float4*>(p.part + ((slot * kBc + r) * 2 + which) * D + c);
                const float4 a = __ldcg(from), b = __ldcg(from + 1);
                acc[0] += a.x, acc[1] += a.y, acc[2] += a.z, acc[3] += a.w;
                acc[4] += b.x, acc[5] += b.y, acc[6] += b.z, acc[7] += b.w;
            }
            __nv_bfloat16* dst = which ? p.dk + head * p.dks[0] + static_cast<int64_t>(key0 + r) * p.dks[1]
                                       : p.dv + head * p.dvs[0] + static_cast<int64_t>(key0 + r) * p.dvs[1];
            *reinterpret_cast<uint4*>(dst + c) = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                                                            pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
        }
        return;
    }
    // Two rows' parts a thread, both under way before the search for their tokens' sequences.
    constexpr int kRowsCta = 256 / kVecs;
    const int64_t rows = static_cast<int64_t>(q.Hq) * q.Nq;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x - cut_ctas) * (2 * kRowsCta) + threadIdx.x / kVecs;
    const int part = threadIdx.x % kVecs;
    float4 a[2], b[2];
    int tok[2], h[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int64_t row = row0 + u * kRowsCta;
        tok[u] = -1;
        if (row < rows) {
            tok[u] = static_cast<int>(row / q.Hq);
            h[u] = static_cast<int>(row - static_cast<int64_t>(tok[u]) * q.Hq);
            const int hk = h[u] / q.G;
            const float4* z = reinterpret_cast<const float4*>(p.dq_acc + ((static_cast<int64_t>(hk) * q.Nq + tok[u]) * q.G + (h[u] - hk * q.G)) * D);
            a[u] = __ldcs(z + 2 * part);
            b[u] = __ldcs(z + 2 * part + 1);
        }
    }
    auto round_row = [&](int u) {
        reinterpret_cast<uint4*>(q.dq + h[u] * q.dqs[0] + tok[u] * q.dqs[1])[part] =
            make_uint4(pack_bf16x2(a[u].x, a[u].y), pack_bf16x2(a[u].z, a[u].w), pack_bf16x2(b[u].x, b[u].y), pack_bf16x2(b[u].z, b[u].w));
    };
    // Up to 256 offsets the CTA looks through all of them for its tokens at once (it has 64 rows at most; bit i is token t0 + i).
    // So it does where offsets fall (behind the last sequence of a padded batch, say), which cannot be searched.  Looked
    // through and searched, calls at 24 heads of 128: 24 texts, 20588 tokens, 740 and 752 us; 256 sequences in 40000 rows, half of
    // them padding, 459 and 495; 2048 in as many 938 (eight goes) and 897.
    if (p.R <= 256 || *p.falls != 0) {
        __shared__ unsigned long long s_in;
        if (threadIdx.x == 0) s_in = 0;
        __syncthreads();
        static_assert(2 * kRowsCta <= 64, "a bit for each token");
        const int t0 = static_cast<int>(static_cast<int64_t>(blockIdx.x - cut_ctas) * (2 * kRowsCta) / q.Hq);
        unsigned long long bits = 0;
        for (int s = threadIdx.x; s < p.R; s += 256) {
            const int from = max(__ldg(p.q_starts + s), t0), to = min(__ldg(p.q_starts + s + 1), t0 + 64);
            if (from < to) bits |= (~0ull >> (64 - (to - from))) << (from - t0);
        }
        if (bits != 0) atomicOr(&s_in, bits);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (tok[u] >= 0 && (s_in >> (tok[u] - t0) & 1)) round_row(u);
        return;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        if (tok[u] < 0) return;
        int lo = 0, hi = p.R;  // the last sequence that begins at or before the token
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (__ldg(p.q_starts + mid) <= tok[u]) lo = mid + 1;
            else hi = mid;
        }
        if (lo == 0 || tok[u] >= __ldg(p.q_starts + lo)) continue;
        round_row(u);
    }
}

}  // namespace elsattn
