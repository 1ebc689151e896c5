// C ABI of attention over a shared prefix and the requests' own keys: argument
// checks, the cut of the prefix into items, TMA descriptors, launches.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "../../include/exact_attn.h"
#include "api_common.h"
#include "attn_prefix_kernel.cuh"

namespace elsattn {
namespace {

struct PrefixShape {
    int R, Hq, Hk, T, P, C, d;
};

int check_shape(const PrefixShape& s) {
    if (s.R < 1 || s.Hq < 1 || s.Hk < 1 || s.T < 1 || s.P < 0 || s.C < 0) return ATTN_ERR_INVALID_ARG;
    if (s.P == 0 && s.C == 0) return ATTN_ERR_INVALID_ARG;
    if (s.Hq % s.Hk != 0) return ATTN_ERR_INVALID_ARG;
    if (static_cast<long long>(s.R) * s.Hq >= kRoundedSizeLimit ||
        static_cast<long long>(s.R) * s.Hq * s.T >= kRoundedSizeLimit || s.P >= kRoundedSizeLimit || s.C >= kRoundedSizeLimit)
        return ATTN_ERR_INVALID_ARG;
    if (s.d != 64 && s.d != 128) return ATTN_ERR_UNSUPPORTED;
    // the kernels count tiles and steps of work in 32 bits (2^31 of them would not fit device memory)
    const double heads = s.Hk, blocks = std::ceil(static_cast<double>(s.Hq / s.Hk) * s.T / 8);
    if (heads * (static_cast<double>(s.P) / kBc + 1) >= 1073741824.0 ||
        s.R * heads * blocks * (static_cast<double>(s.C) / kOwnStep + kPfxItemCost + 1) >= 1073741824.0)
        return ATTN_ERR_INVALID_ARG;
    return ATTN_OK;
}

// What the cut of the prefix costs besides its tiles, in the kernel's units of
// work (a tile of 128 keys is 4, about 1.6 us with two query tiles): a piece's
// start and end (3 us: its rows, the pipeline's fill, O out), and a partial row
// written and read back (1 KB at 6 TB/s).
constexpr double kPlanPiece = 8.0;
constexpr double kPlanRow = 4.2e-4;

// The own-keys kernel is bound by HBM and the prefix, with many rows, by the
// tensor core.  The former reads 5.9 TB/s on all SMs, 5.3 on 96 and 4.4 on 76, so about 5 on 88, which is what it gets
// where there is a prefix to run beside it; a step of 16 keys of 128 then takes
// 1 / 976 of a prefix tile's time.  Measured, own kernel on all SMs -> on 88: 64 requests on
// 16384 keys, up to 1024 own 60.4 -> 53.7 us (96 SMs 57.4, 80 52.1, 72 55.4 us), with 1024 own each 78.9 -> 77.3
// (72.0, 80.9, 88.3) us, 256 on 65536 246.6 -> 239 us.  Not where the own keys could take
// more than about five times the prefix's time (the capacity is what the host knows).
constexpr int kBesideSms = 88;
constexpr int kBesideLead = 1074;          // 2^20 / 976
constexpr double kBesideLeast = 4096.0;    // own steps (6 us)
constexpr double kBesideMost = 5750.0;     // own steps for a prefix tile of every SM: 5 x 1150

// Sizes that follow from the shape, and the cut of the prefix into the number
// of stretches with the least estimated time: items in whole waves, each its
// tiles and its pieces, and the partial rows.
void lay_out(PrefixParams& p, const PrefixShape& s, int num_sms) {
    p.R = s.R;
    p.T = s.T;
    p.Hk = s.Hk;
    p.G = s.Hq / s.Hk;
    p.GT = p.G * s.T;
    p.P = s.P;
    p.C = s.C;
    p.ptiles = (s.P + kBc - 1) / kBc;
    p.qrows = p.GT <= kBr ? kBr / p.GT * p.GT : kBr;
    p.pblocks = static_cast<int>((static_cast<int64_t>(s.R) * p.GT + 2 * p.qrows - 1) / (2 * p.qrows));
    p.oblocks = (p.GT + 2 * p.qrows - 1) / (2 * p.qrows);
    p.orows = p.GT < 2 * p.qrows ? p.GT : 2 * p.qrows;
    // Own keys of few rows a request and key head: a kernel of their own (see there), with row
    // blocks of whole heads of the group.  Its warps: as many as there can be steps for, up to kOwnWarps an SM.
    // Beside a prefix, up to one sequence an SM are items of the prefix kernel: that takes the GPU about as
    // long and saves the host a launch (a call from the host on the first shape below: 19 us, 25 with the own kernel).
    // GPU time of calls in a replayed graph, as items and with the own kernel: 8 requests x 8 heads on 1000 prefix keys, up to 64
    // own, 13.5 and 12.9 us; 128 x 1 (16 query heads) on 8192, up to 256 own, 26.4 and 29.1 us; but 16 x 8 on 1000 with
    // 40 own each 15.9 and 14.0 us, and near the boundary on long caches (19 x 8, 8192 own keys) 110.1 and 106.6 us.
    p.workers = 0;
    const bool few = s.P > 0 && static_cast<int64_t>(s.R) * s.Hk <= num_sms;
    if (s.C > 0 && !few && s.T <= kOwnRows && (p.GT <= kOwnRows || (p.GT <= kOwnMostRows && s.C <= kOwnMostKeys))) {
        const int heads = kOwnRows / s.T < p.G ? kOwnRows / s.T : p.G;
        p.oblocks = (p.G + heads - 1) / heads;
        p.orows = heads * s.T;
        const int64_t steps = static_cast<int64_t>(s.R) * s.Hk * p.oblocks * ((s.C + kOwnStep - 1) / kOwnStep);
        const int64_t ctas = (steps + kOwnWarps - 1) / kOwnWarps;
        p.workers = static_cast<int>(ctas < num_sms ? ctas : num_sms) * kOwnWarps;
    }
    p.psegs = 0;
    p.pitems = 0;
    p.by_head = p.run_per = 1;
    p.run_len = p.even_base = p.even_rem = 0;
    p.early = p.lead = 0;
    if (p.ptiles > 0) {
        // (in floating point: the quotients are small and this is on every call's path)
        const double line = static_cast<double>(s.Hk) * p.ptiles, blocks = p.pblocks, sms = num_sms, heads = s.Hk;
        const int most = static_cast<int>(std::fmin(line, std::fmax(8.0, std::floor(2.0 * sms / blocks))));
        const double row = kPlanRow * s.R * p.GT;
        double best = 0;
        int rest = 0;  // n modulo the key heads
        for (int n = 1; n <= most; ++n) {
            rest = rest + 1 == s.Hk ? 0 : rest + 1;
            // the most pieces of a stretch: key heads' borders fall on stretches' where they can
            const double pieces = rest == 0 ? 1.0 : std::ceil(heads / n) + 1.0;
            const double cost = std::ceil(blocks * n / sms) * (std::ceil(line / n) * kPfxTileCost + pieces * kPlanPiece) + row * (n + heads);
            if (n == 1 || cost < best) {
                best = cost;
                p.psegs = n;
            }
        }
        p.pitems = p.pblocks * p.psegs;
        p.by_head = p.psegs % s.Hk == 0;
        p.run_len = p.by_head ? p.ptiles : p.ptiles * s.Hk;
        p.run_per = p.by_head ? p.psegs / s.Hk : p.psegs;
        p.even_base = p.run_len / p.run_per;
        p.even_rem = p.run_len % p.run_per;
        // Side by side: the own-keys kernel leaves SMs to the prefix, whose first stretches start at once and are longer.
        const double own_steps = p.workers == 0 ? 0.0 : static_cast<double>(s.R) * s.Hk * p.oblocks * ((s.C + kOwnStep - 1) / kOwnStep);
        if (p.pitems <= num_sms && p.workers > kBesideSms * kOwnWarps && own_steps >= kBesideLeast && line >= 3.0 * p.psegs &&
            own_steps <= kBesideMost * line * blocks / sms) {
            p.workers = kBesideSms * kOwnWarps;
            const int beside = (num_sms - kBesideSms) / p.pblocks;  // stretches whose CTAs start at once
            p.early = p.by_head ? beside / s.Hk : beside;
            if (p.early >= p.run_per) p.early = p.run_per - 1;
            p.lead = s.d == 128 ? kBesideLead : kBesideLead * 3 / 4;
        }
    }
}

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// Workspace: [R + 1 int][log-sum-exp of the partial rows][partial rows].
struct PrefixSpace {
    size_t start, lse, rows, bytes;
    int64_t own_first;
    PrefixSpace(const PrefixParams& p, int d, int num_sms) {
        const int grid = p.workers > 0 ? p.workers : num_sms;  // who may have a piece of a sequence
        own_first = p.psegs == 0 ? 0 : static_cast<int64_t>(p.psegs + (p.by_head ? 0 : p.Hk - 1)) * p.R * p.GT;
        const int64_t own = p.C > 0 ? (static_cast<int64_t>(p.R) * p.Hk * p.oblocks + grid) * p.orows : 0;
        start = 0;
        lse = align256((static_cast<size_t>(p.R) + 1) * sizeof(int));
        rows = lse + align256(static_cast<size_t>(own_first + own) * sizeof(float));
        bytes = rows + static_cast<size_t>(own_first + own) * d * sizeof(float);
    }
};

template <int D>
int launch(DeviceState& dev, const CUtensorMap (&maps)[6], const PrefixParams& p, cudaStream_t stream) {
    auto kernel = attn_prefix_kernel<D>;
    constexpr int smem = PrefixSmem<D>::kBytes;
    bool& configured = dev.prefix_smem_configured[0][D == 128];
    cudaError_t e;
    if (!configured) {
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
            return cuda_fail(e);
        configured = true;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    if (p.workers > 0) {
        auto own = attn_prefix_own_kernel<D>;
        constexpr int own_smem = OwnSmem<D>::kBytes;
        bool& own_configured = dev.prefix_smem_configured[1][D == 128];
        if (!own_configured) {
            if ((e = cudaFuncSetAttribute(own, cudaFuncAttributeMaxDynamicSharedMemorySize, own_smem)) != cudaSuccess)
                return cuda_fail(e);
            own_configured = true;
        }
        own<<<p.workers / kOwnWarps, kOwnWarps * 32, own_smem, stream>>>(maps[1], maps[4], maps[5], p);
        if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e);
        // the prefix kernel is a programmatic dependent: its CTAs start as the SMs become free
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    if (p.workers == 0 || p.pitems > 0) {
        // with own items, a CTA per SM (their cut counts on it); else no more than there are items
        const bool own_items = p.C > 0 && p.workers == 0;
        const int grid = !own_items && p.pitems < dev.num_sms ? p.pitems : dev.num_sms;
        cfg.gridDim = dim3(static_cast<unsigned>(grid));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        if ((e = cudaLaunchKernelEx(&cfg, kernel, maps[0], maps[1], maps[2], maps[3], maps[4], maps[5], p)) != cudaSuccess)
            return cuda_fail(e);
    }
    // A row's pieces are dealt to as many warps (1, 2, 4, 8) as there are pieces for and as the SMs hold at
    // once (32 each).  Whole calls: 2048 rows of 19 pieces 32.8 us with the two warps this gives (one 35.0, eight
    // 37.3 us); 256 rows of 19 pieces 24.5 us with eight (one 28.8 us); 8192 rows of 6 195 us with one (eight 220 us).
    const int64_t rows = static_cast<int64_t>(p.R) * p.Hk * p.GT;
    const int pieces = (p.psegs + p.Hk - 1) / p.Hk + (p.C > 0 ? 1 : 0);  // about
    int warps = 1;
    while (warps < 8 && warps < pieces && rows * warps * 2 <= 32ll * dev.num_sms) warps *= 2;
    cfg.gridDim = dim3(static_cast<unsigned>((rows * warps + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto combine = warps == 8 ? attn_prefix_combine_kernel<D, 8> : warps == 4 ? attn_prefix_combine_kernel<D, 4>
                   : warps == 2 ? attn_prefix_combine_kernel<D, 2> : attn_prefix_combine_kernel<D, 1>;
    if ((e = cudaLaunchKernelEx(&cfg, combine, p, dev.num_sms)) != cudaSuccess) return cuda_fail(e);
    return ATTN_OK;
}

}  // namespace
}  // namespace elsattn

using namespace elsattn;

extern "C" size_t attn_fwd_prefix_workspace_bytes(int R, int Hq, int Hk, int T, int P, int C, int d) {
    const PrefixShape s{R, Hq, Hk, T, P, C, d};
    if (check_shape(s) != ATTN_OK) return 0;
    DeviceState* dev = nullptr;
    if (device_state(&dev) != ATTN_OK) return 0;
    PrefixParams p;
    lay_out(p, s, dev->num_sms);
    return PrefixSpace(p, d, dev->num_sms).bytes;
}

extern "C" int attn_fwd_prefix(const void* Q, const int64_t* q_strides, const void* Kp, const int64_t* kp_strides,
                               const void* Vp, const int64_t* vp_strides, const void* Ko, const int64_t* ko_strides,
                               const void* Vo, const int64_t* vo_strides, const int32_t* own_lens, void* O,
                               const int64_t* o_strides, float* LSE, int R, int Hq, int Hk, int T, int P, int C, int d,
                               float scale, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    const PrefixShape s{R, Hq, Hk, T, P, C, d};
    int st = check_shape(s);
    if (st != ATTN_OK) return st;
    if (!Q || !O || !LSE || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
    if ((P > 0 && (!Kp || !Vp)) || (C > 0 && (!Ko || !Vo || !own_lens))) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(Q) || !aligned16(O) || (reinterpret_cast<uintptr_t>(LSE) & 3u) != 0 ||
        (P > 0 && (!aligned16(Kp) || !aligned16(Vp))) ||
        (reinterpret_cast<uintptr_t>(own_lens) & 3u) != 0 || (C > 0 && (!aligned16(Ko) || !aligned16(Vo))))
        return ATTN_ERR_MISALIGNED;
    if (!workspace) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(workspace)) return ATTN_ERR_MISALIGNED;
    PrefixParams p;
    int64_t kp[2], vp[2], ko[3], vo[3];
    const int64_t rows_dims[3] = {R, Hq, T}, pre_dims[2] = {Hk, P}, own_dims[3] = {R, Hk, C};
    if ((st = take_view(p.qs, q_strides, rows_dims, d)) != ATTN_OK ||
        (st = take_view(p.os, o_strides, rows_dims, d)) != ATTN_OK ||
        (P > 0 && ((st = take_view(kp, kp_strides, pre_dims, d)) != ATTN_OK ||
                   (st = take_view(vp, vp_strides, pre_dims, d)) != ATTN_OK)) ||
        (C > 0 && ((st = take_view(ko, ko_strides, own_dims, d)) != ATTN_OK ||
                   (st = take_view(vo, vo_strides, own_dims, d)) != ATTN_OK)))
        return st;
    DeviceState* dev = nullptr;
    if ((st = device_state(&dev)) != ATTN_OK) return st;
    lay_out(p, s, dev->num_sms);
    const PrefixSpace space(p, d, dev->num_sms);
    if (workspace_bytes < space.bytes) return ATTN_ERR_INVALID_ARG;
    CUtensorMap maps[6] = {};  // Q by tiles of the prefix, Q by requests; Kp, Vp; Ko, Vo
    const void* pre[2] = {Kp, Vp};
    const void* own[2] = {Ko, Vo};
    const int64_t *pre_st[2] = {kp, vp}, *own_st[2] = {ko, vo};
    for (int i = 0; i < 2; ++i) {
        if (P > 0) {
            const uint64_t e[3] = {static_cast<uint64_t>(d), static_cast<uint64_t>(P), static_cast<uint64_t>(Hk)};
            const uint64_t b[2] = {static_cast<uint64_t>(pre_st[i][1]) * 2, static_cast<uint64_t>(pre_st[i][0]) * 2};
            const uint32_t box[3] = {64, kBc, 1};
            if ((st = encode_bf16_map(&maps[2 + i], pre[i], 3, e, b, box)) != ATTN_OK) return st;
        }
        if (C > 0) {
            const uint64_t e[4] = {static_cast<uint64_t>(d), static_cast<uint64_t>(C), static_cast<uint64_t>(Hk),
                                   static_cast<uint64_t>(R)};
            const uint64_t b[3] = {static_cast<uint64_t>(own_st[i][2]) * 2, static_cast<uint64_t>(own_st[i][1]) * 2,
                                   static_cast<uint64_t>(own_st[i][0]) * 2};
            const uint32_t box[4] = {64, static_cast<uint32_t>(p.workers > 0 ? kOwnStep : kPfxOwnBox), 1, 1};
            if ((st = encode_bf16_map(&maps[4 + i], own[i], 4, e, b, box)) != ATTN_OK) return st;
        }
    }
    if (p.GT <= kBr) {
        const uint64_t e[5] = {static_cast<uint64_t>(d), static_cast<uint64_t>(T), static_cast<uint64_t>(p.G),
                               static_cast<uint64_t>(Hk), static_cast<uint64_t>(R)};
        const uint64_t b[4] = {static_cast<uint64_t>(p.qs[2]) * 2, static_cast<uint64_t>(p.qs[1]) * 2,
                               static_cast<uint64_t>(p.qs[1]) * p.G * 2, static_cast<uint64_t>(p.qs[0]) * 2};
        const uint32_t tile[5] = {64, static_cast<uint32_t>(T), static_cast<uint32_t>(p.G), 1,
                                  static_cast<uint32_t>(p.qrows / p.GT)};
        const uint32_t one[5] = {64, static_cast<uint32_t>(T), static_cast<uint32_t>(p.workers > 0 ? p.orows / T : p.G), 1, 1};
        if ((P > 0 && (st = encode_bf16_map(&maps[0], Q, 5, e, b, tile)) != ATTN_OK) ||
            (C > 0 && (st = encode_bf16_map(&maps[1], Q, 5, e, b, one)) != ATTN_OK))
            return st;
    }
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.q = static_cast<const __nv_bfloat16*>(Q);
    p.o = static_cast<__nv_bfloat16*>(O);
    p.lse = LSE;
    p.lens = own_lens;
    p.own_start = reinterpret_cast<int*>(ws + space.start);
    p.part_lse = reinterpret_cast<float*>(ws + space.lse);
    p.part_o = reinterpret_cast<float*>(ws + space.rows);
    p.own_first = space.own_first;
    p.error_word = dev->error_word;
    p.timeout_ns = kDefaultTimeoutNs;
    // A negative scale runs as |scale| on the negated scores; a zero scale as the
    // smallest normal factor in the exponents and 0 in the running maximum (as
    // attn_fwd does): every visible key's weight is then exactly 1.
    p.negate_scores = scale < 0.f ? 1u : 0u;
    p.scale_log2 = scale == 0.f ? FLT_MIN : std::fabs(scale) * 1.4426950408889634f;
    p.max_scale_log2 = scale == 0.f ? 0.f : p.scale_log2;
    return d == 64 ? launch<64>(*dev, maps, p, stream) : launch<128>(*dev, maps, p, stream);
}
