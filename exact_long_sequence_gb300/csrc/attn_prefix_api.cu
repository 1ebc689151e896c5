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
    if (static_cast<long long>(s.R) * s.Hq >= (1LL << 31) || static_cast<long long>(s.R) * s.Hq * s.T >= (1LL << 31))
        return ATTN_ERR_INVALID_ARG;
    if (s.d != 64 && s.d != 128) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

// Sizes that follow from the shape, and the cut of the prefix: the number of
// segments with the least estimated time, in the units of the kernel's own
// work (items in whole waves, each its tiles and a constant), plus what a
// further segment costs the combine kernel.
void lay_out(PrefixParams& p, const PrefixShape& s, int num_sms) {
    p.R = s.R;
    p.T = s.T;
    p.Hk = s.Hk;
    p.G = s.Hq / s.Hk;
    p.GT = p.G * s.T;
    p.P = s.P;
    p.C = s.C;
    p.ptiles = (s.P + kBc - 1) / kBc;
    p.pblocks = static_cast<int>((static_cast<int64_t>(s.R) * p.GT + 2 * kBr - 1) / (2 * kBr));
    p.oblocks = (p.GT + 2 * kBr - 1) / (2 * kBr);
    p.orows = p.GT < 2 * kBr ? p.GT : 2 * kBr;
    p.psegs = 0;
    p.seg_tiles = 1;
    p.pitems = 0;
    if (p.ptiles > 0) {
        const int64_t units = static_cast<int64_t>(s.Hk) * p.pblocks;
        int64_t most = 2 * num_sms / units;
        if (most < 8) most = 8;
        if (most > p.ptiles) most = p.ptiles;
        double best = 0;
        for (int64_t n = 1; n <= most; ++n) {
            const int64_t tiles = (p.ptiles + n - 1) / n;
            const int64_t waves = (units * n + num_sms - 1) / num_sms;
            const double cost = static_cast<double>(waves) * (kPfxItemCost + tiles * kPfxTileCost) + 0.25 * n;
            if (n == 1 || cost < best) {
                best = cost;
                p.seg_tiles = static_cast<int>(tiles);
            }
        }
        p.psegs = (p.ptiles + p.seg_tiles - 1) / p.seg_tiles;
        p.pitems = static_cast<int>(units * p.psegs);
    }
}

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// Workspace: [R + 1 int64][log-sum-exp of the partial rows][partial rows].
struct PrefixSpace {
    size_t start, lse, rows, bytes;
    int64_t own_first;
    PrefixSpace(const PrefixParams& p, int d, int grid) {
        own_first = static_cast<int64_t>(p.psegs) * p.Hk * p.R * p.GT;
        const int64_t own = p.C > 0 ? (static_cast<int64_t>(p.R) * p.Hk * p.oblocks + grid) * p.orows : 0;
        start = 0;
        lse = align256(static_cast<size_t>(p.R + 1) * sizeof(int64_t));
        rows = lse + align256(static_cast<size_t>(own_first + own) * sizeof(float));
        bytes = rows + static_cast<size_t>(own_first + own) * d * sizeof(float);
    }
};

// Strides of a view in elements; nullptr: contiguous.  TMA takes strides of a
// multiple of 16 bytes below 2^40; an axis of one is never stepped.
template <int N>
int take_view(int64_t (&out)[N], const int64_t* given, const int64_t (&dims)[N], int64_t inner) {
    int64_t dense = inner;
    for (int i = N - 1; i >= 0; --i) {
        out[i] = dense;
        if (given && dims[i] > 1) {
            out[i] = given[i];
            if (out[i] % 8 != 0) return ATTN_ERR_MISALIGNED;
            if (out[i] <= 0 || out[i] >= (1LL << 39)) return ATTN_ERR_INVALID_ARG;
        }
        dense *= dims[i];
    }
    return ATTN_OK;
}

template <int D>
int launch(DeviceState& dev, const CUtensorMap (&maps)[4], const PrefixParams& p, cudaStream_t stream) {
    auto kernel = attn_prefix_kernel<D>;
    constexpr int smem = PrefixSmem<D>::kBytes;
    bool& configured = dev.prefix_smem_configured[D == 128];
    cudaError_t e;
    if (!configured) {
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
            return cuda_fail(e);
        configured = true;
    }
    kernel<<<dev.num_sms, kThreads, smem, stream>>>(maps[0], maps[1], maps[2], maps[3], p);
    if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e);
    // one warp a row, or eight where there are few rows and many pieces to merge
    const int64_t rows = static_cast<int64_t>(p.R) * p.Hk * p.GT;
    const bool wide = rows < 8 * static_cast<int64_t>(dev.num_sms);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(wide ? rows : (rows + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto combine = wide ? attn_prefix_combine_kernel<D, 8> : attn_prefix_combine_kernel<D, 1>;
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
        (C > 0 && (!aligned16(Ko) || !aligned16(Vo) || (reinterpret_cast<uintptr_t>(own_lens) & 3u) != 0)))
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
    CUtensorMap maps[4] = {};
    const void* pre[2] = {Kp, Vp};
    const void* own[2] = {Ko, Vo};
    const int64_t *pre_st[2] = {kp, vp}, *own_st[2] = {ko, vo};
    for (int i = 0; i < 2; ++i) {
        if (P > 0) {
            const uint64_t e[3] = {static_cast<uint64_t>(d), static_cast<uint64_t>(P), static_cast<uint64_t>(Hk)};
            const uint64_t b[2] = {static_cast<uint64_t>(pre_st[i][1]) * 2, static_cast<uint64_t>(pre_st[i][0]) * 2};
            if ((st = encode_bf16_map(&maps[i], pre[i], 3, e, b, kBc)) != ATTN_OK) return st;
        }
        if (C > 0) {
            const uint64_t e[4] = {static_cast<uint64_t>(d), static_cast<uint64_t>(C), static_cast<uint64_t>(Hk),
                                   static_cast<uint64_t>(R)};
            const uint64_t b[3] = {static_cast<uint64_t>(own_st[i][2]) * 2, static_cast<uint64_t>(own_st[i][1]) * 2,
                                   static_cast<uint64_t>(own_st[i][0]) * 2};
            if ((st = encode_bf16_map(&maps[2 + i], own[i], 4, e, b, kPfxOwnBox)) != ATTN_OK) return st;
        }
    }
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.q = static_cast<const __nv_bfloat16*>(Q);
    p.o = static_cast<__nv_bfloat16*>(O);
    p.lse = LSE;
    p.lens = C > 0 ? own_lens : nullptr;
    p.own_start = reinterpret_cast<int64_t*>(ws + space.start);
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
