// C ABI of attention over packed sequences and over a paged cache: argument
// checks, the cut of the work, TMA descriptors, launches.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "../../include/exact_attn.h"
#include "api_common.h"
#include "attn_packed_kernel.cuh"

namespace elsattn {
namespace {

// K and V that the CTAs read at a time: the line has a stretch a CTA for each so many bytes, up to kMostTurns (documents of
// 3001 to 16384 tokens, 32 heads of 8, with 30, 64, 128 and 1000 MB: 2170, 2146, 2142 and 2175 us).
constexpr double kTurnBytes = 128e6;
constexpr int kMostTurns = 8;

// Up to so many keys in all (of a request's cache: the host knows no lengths, but these bounds), no unit is cut and the launch that
// merges pieces is left out.  Cut and merged, and like this (causal, d = 128, replayed from a graph): 4 sequences of 64 tokens at
// 8 heads 10.8 and 9.5 us, one of 600 19.0 and 15.8, at 32 heads of 8 26.1 and 17.8; with more keys few heads lose (1200 at 8 heads
// 22.8 and 24.0, 2400 33.9 and 36.5), and the kernel decides by the lengths (line_whole).
constexpr int kWholeKeys = 640;

// Sizes that follow from the shape.  tokens, keys: most of a sequence; kv_bytes: of K and V together.
void lay_out(PackedParams& p, int Hq, int Hk, int64_t tokens, int64_t keys, double kv_bytes, int num_sms) {
    p.whole = keys <= kWholeKeys;
    p.Hk = Hk;
    p.G = Hq / Hk;
    p.tile_tokens = kBr / p.G;
    p.qrows = p.tile_tokens * p.G;
    const int64_t rows = tokens * p.G;
    p.orows = rows < 2 * p.qrows ? static_cast<int>(rows) : 2 * p.qrows;
    int turns = static_cast<int>(std::fmin(std::ceil(kv_bytes / kTurnBytes), kMostTurns));
    if (turns < 1) turns = 1;
    while (turns > 1 && num_sms * turns > kPkMostStretches) --turns;
    p.stretches = num_sms * turns;  // (an SM count above kPkMostStretches there is not: device_state takes sm_103 only)
}

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// Workspace: [stretches] cuts, log-sum-exp of the partial rows, partial rows.
struct PackedSpace {
    size_t lse, rows, bytes;
    PackedSpace(const PackedParams& p, int d) {
        const size_t part = p.whole ? 0 : 2 * static_cast<size_t>(p.stretches) * p.orows;
        lse = align256(p.stretches * sizeof(PackedCut));
        rows = lse + align256(part * sizeof(float));
        bytes = rows + part * d * sizeof(float);
    }
};

int check_heads(int Hq, int Hk, int d) {
    if (Hq < 1 || Hk < 1 || Hq % Hk != 0) return ATTN_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    if (Hq / Hk > kPkMostGroup) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

int check_packed(int R, int Nq, int Nk, int Hq, int Hk, int d) {
    if (R < 1 || Nq < 1 || Nk < 1) return ATTN_ERR_INVALID_ARG;
    const int st = check_heads(Hq, Hk, d);
    if (st != ATTN_OK) return st;
    if (static_cast<long long>(Hq) * Nq >= kRoundedSizeLimit || static_cast<long long>(Hk) * Nk >= kRoundedSizeLimit ||
        R >= kRoundedSizeLimit)
        return ATTN_ERR_INVALID_ARG;
    return ATTN_OK;
}

int check_tree(int R, int Hq, int Hk, int T, int pages, int page_size, int table_pages, int d) {
    if (R < 1 || T < 1 || pages < 1 || page_size < 1 || table_pages < 1) return ATTN_ERR_INVALID_ARG;
    const int st = check_heads(Hq, Hk, d);
    if (st != ATTN_OK) return st;
    if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) != 0) return ATTN_ERR_UNSUPPORTED;
    if (static_cast<long long>(R) * Hq >= kRoundedSizeLimit || static_cast<long long>(R) * Hq * T >= kRoundedSizeLimit ||
        static_cast<long long>(table_pages) * page_size >= kRoundedSizeLimit || pages >= kRoundedSizeLimit)
        return ATTN_ERR_INVALID_ARG;
    return ATTN_OK;
}

void take_scale(PackedParams& p, float scale) {
    // A negative scale runs as |scale| on the negated scores; a zero scale as the
    // smallest normal factor in the exponents and 0 in the running maximum (as
    // attn_fwd does): every visible key's weight is then exactly 1.
    p.negate_scores = scale < 0.f ? 1u : 0u;
    p.scale_log2 = scale == 0.f ? FLT_MIN : std::fabs(scale) * 1.4426950408889634f;
    p.max_scale_log2 = scale == 0.f ? 0.f : p.scale_log2;
}

template <int D, bool PAGED>
int launch(DeviceState& dev, const CUtensorMap (&maps)[5], const PackedParams& p, cudaStream_t stream) {
    auto kernel = attn_packed_kernel<D, PAGED>;
    constexpr int smem = PackedSmem<D>::kBytes;
    bool& configured = dev.packed_smem_configured[PAGED][D == 128];
    cudaError_t e;
    if (!configured) {
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
            return cuda_fail(e);
        configured = true;
    }
    // The first launch is a plain one.  As a programmatic dependent it would wait for the grid before it only, and
    // where the caller's own grid is one that does not wait for those before, these could still run.
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.gridDim = dim3(static_cast<unsigned>(dev.num_sms));
    cfg.blockDim = dim3(kPkThreads);
    cfg.dynamicSmemBytes = smem;
    if ((e = cudaLaunchKernelEx(&cfg, kernel, maps[0], maps[1], maps[2], maps[3], maps[4], p)) != cudaSuccess) return cuda_fail(e);
    if (p.whole) return ATTN_OK;
    // The merge sets up beside the end of the first kernel, and waits for it.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.dynamicSmemBytes = 0;
    cfg.gridDim = dim3(static_cast<unsigned>(4 * dev.num_sms));
    cfg.blockDim = dim3(256);
    if ((e = cudaLaunchKernelEx(&cfg, attn_packed_combine_kernel<D>, p)) != cudaSuccess) return cuda_fail(e);
    return ATTN_OK;
}

// The kernels' memory and status, and the launch for d.
template <bool PAGED>
int run(DeviceState& dev, const CUtensorMap (&maps)[5], PackedParams& p, int d, float scale, void* workspace, cudaStream_t stream) {
    const PackedSpace space(p, d);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.cuts = reinterpret_cast<PackedCut*>(ws);
    p.part_lse = reinterpret_cast<float*>(ws + space.lse);
    p.part_o = reinterpret_cast<float*>(ws + space.rows);
    p.error_word = dev.error_word;
    p.timeout_ns = kDefaultTimeoutNs;
    if (const uint64_t t = take_armed_timeout()) {  // (test hook)
        p.timeout_ns = t;
        p.withhold_first_q = 1u;
    }
    take_scale(p, scale);
    return d == 64 ? launch<64, PAGED>(dev, maps, p, stream) : launch<128, PAGED>(dev, maps, p, stream);
}

// Q as [request][token][key head][head of the group][d], in boxes of a query tile.
int encode_q(CUtensorMap* map, const void* Q, const PackedParams& p, int d, int R, int tokens, int64_t req, int64_t head, int64_t token) {
    const uint64_t e[5] = {static_cast<uint64_t>(d), static_cast<uint64_t>(p.G), static_cast<uint64_t>(p.Hk),
                           static_cast<uint64_t>(tokens), static_cast<uint64_t>(R)};
    const uint64_t b[4] = {static_cast<uint64_t>(head) * 2, static_cast<uint64_t>(head) * p.G * 2, static_cast<uint64_t>(token) * 2,
                           static_cast<uint64_t>(req) * 2};
    const uint32_t box[5] = {64, static_cast<uint32_t>(p.G), 1, static_cast<uint32_t>(p.tile_tokens), 1};
    return encode_bf16_map(map, Q, 5, e, b, box);
}

}  // namespace
}  // namespace elsattn

using namespace elsattn;

extern "C" size_t attn_fwd_packed_workspace_bytes(int R, int Nq, int Nk, int Hq, int Hk, int d) {
    if (check_packed(R, Nq, Nk, Hq, Hk, d) != ATTN_OK) return 0;
    DeviceState* dev = nullptr;
    if (device_state(&dev) != ATTN_OK) return 0;
    PackedParams p{};
    lay_out(p, Hq, Hk, Nq, Nk, 4.0 * Nk * Hk * d, dev->num_sms);
    return PackedSpace(p, d).bytes;
}

extern "C" int attn_fwd_packed(const void* Q, const int64_t* q_strides, const void* K, const int64_t* k_strides, const void* V,
                               const int64_t* v_strides, const int32_t* q_starts, const int32_t* k_starts, void* O,
                               const int64_t* o_strides, float* LSE, int R, int Nq, int Nk, int Hq, int Hk, int d, int causal,
                               float scale, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    int st = check_packed(R, Nq, Nk, Hq, Hk, d);
    if (st != ATTN_OK) return st;
    if (!Q || !K || !V || !q_starts || !k_starts || !O || !LSE || !workspace || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O) || !aligned16(workspace) ||
        ((reinterpret_cast<uintptr_t>(LSE) | reinterpret_cast<uintptr_t>(q_starts) | reinterpret_cast<uintptr_t>(k_starts)) & 3u) != 0)
        return ATTN_ERR_MISALIGNED;
    PackedParams p{};
    int64_t qs[2], ks[2], vs[2], os[2];
    const int64_t q_dims[2] = {Hq, Nq}, k_dims[2] = {Hk, Nk};
    if ((st = take_view(qs, q_strides, q_dims, d)) != ATTN_OK || (st = take_view(os, o_strides, q_dims, d)) != ATTN_OK ||
        (st = take_view(ks, k_strides, k_dims, d)) != ATTN_OK || (st = take_view(vs, v_strides, k_dims, d)) != ATTN_OK)
        return st;
    DeviceState* dev = nullptr;
    if ((st = device_state(&dev)) != ATTN_OK) return st;
    p.R = R;
    p.Nq = Nq;
    p.Nk = Nk;
    p.causal = causal != 0;
    lay_out(p, Hq, Hk, Nq, Nk, 4.0 * Nk * Hk * d, dev->num_sms);
    if (workspace_bytes < PackedSpace(p, d).bytes) return ATTN_ERR_INVALID_ARG;
    p.q_starts = q_starts;
    p.k_starts = k_starts;
    p.o = static_cast<__nv_bfloat16*>(O);
    p.os[1] = os[0];
    p.os[2] = os[1];
    p.lse = LSE;
    p.ls[1] = Nq;
    CUtensorMap maps[5];
    const void* kv[2] = {K, V};
    const int64_t* kvs[2] = {ks, vs};
    for (int i = 0; i < 2; ++i) {
        const uint64_t e[3] = {static_cast<uint64_t>(d), static_cast<uint64_t>(Nk), static_cast<uint64_t>(Hk)};
        const uint64_t b[2] = {static_cast<uint64_t>(kvs[i][1]) * 2, static_cast<uint64_t>(kvs[i][0]) * 2};
        const uint32_t box[3] = {64, kBc, 1}, tail[3] = {64, kPkTailBox, 1};
        if ((st = encode_bf16_map(&maps[1 + i], kv[i], 3, e, b, box)) != ATTN_OK ||
            (st = encode_bf16_map(&maps[3 + i], kv[i], 3, e, b, tail)) != ATTN_OK)
            return st;
    }
    // (an axis of one request: its stride is never stepped)
    if ((st = encode_q(&maps[0], Q, p, d, 1, Nq, qs[1], qs[0], qs[1])) != ATTN_OK) return st;
    return run<false>(*dev, maps, p, d, scale, workspace, stream);
}

extern "C" size_t attn_fwd_tree_workspace_bytes(int R, int Hq, int Hk, int T, int d) {
    if (check_tree(R, Hq, Hk, T, 1, 16, 1, d) != ATTN_OK) return 0;
    DeviceState* dev = nullptr;
    if (device_state(&dev) != ATTN_OK) return 0;
    PackedParams p{};
    lay_out(p, Hq, Hk, T, 0, 0.0, dev->num_sms);
    p.whole = false;  // (the caches' capacity is not asked for here)
    return PackedSpace(p, d).bytes;
}

extern "C" int attn_fwd_tree(const void* Q, const int64_t* q_strides, const void* Kc, const int64_t* k_strides, const void* Vc,
                             const int64_t* v_strides, const int32_t* page_table, int64_t table_stride, const int32_t* lens,
                             const int32_t* tree_mask, void* O, const int64_t* o_strides, float* LSE, int R, int Hq, int Hk, int T,
                             int pages, int page_size, int table_pages, int d, float scale, void* workspace,
                             size_t workspace_bytes, cudaStream_t stream) {
    int st = check_tree(R, Hq, Hk, T, pages, page_size, table_pages, d);
    if (st != ATTN_OK) return st;
    if (!Q || !Kc || !Vc || !page_table || !lens || !O || !LSE || !workspace || !std::isfinite(scale) || table_stride < 0)
        return ATTN_ERR_INVALID_ARG;
    if (!aligned16(Q) || !aligned16(Kc) || !aligned16(Vc) || !aligned16(O) || !aligned16(workspace) ||
        ((reinterpret_cast<uintptr_t>(LSE) | reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(lens) |
          reinterpret_cast<uintptr_t>(tree_mask)) & 3u) != 0)
        return ATTN_ERR_MISALIGNED;
    PackedParams p{};
    int64_t qs[3], ks[3], vs[3];
    const int64_t q_dims[3] = {R, Hq, T}, k_dims[3] = {pages, Hk, page_size};
    if ((st = take_view(qs, q_strides, q_dims, d)) != ATTN_OK || (st = take_view(p.os, o_strides, q_dims, d)) != ATTN_OK ||
        (st = take_view(ks, k_strides, k_dims, d)) != ATTN_OK || (st = take_view(vs, v_strides, k_dims, d)) != ATTN_OK)
        return st;
    DeviceState* dev = nullptr;
    if ((st = device_state(&dev)) != ATTN_OK) return st;
    p.R = R;
    p.T = T;
    lay_out(p, Hq, Hk, T, static_cast<int64_t>(table_pages) * page_size, 0.0, dev->num_sms);  // (K and V are read once: nothing to keep in L2)
    if (workspace_bytes < PackedSpace(p, d).bytes) return ATTN_ERR_INVALID_ARG;
    p.lens = lens;
    p.table = page_table;
    p.table_stride = table_stride;
    p.mask = reinterpret_cast<const uint32_t*>(tree_mask);
    p.words = (T + 31) / 32;
    while ((1 << p.page_log2) < page_size) ++p.page_log2;
    p.box = page_size < kBc ? page_size : kBc;
    p.pages = pages;
    p.cap = table_pages * page_size;
    p.o = static_cast<__nv_bfloat16*>(O);
    p.lse = LSE;
    p.ls[0] = static_cast<int64_t>(Hq) * T;
    p.ls[1] = T;
    CUtensorMap maps[5];
    const void* kv[2] = {Kc, Vc};
    const int64_t* kvs[2] = {ks, vs};
    for (int i = 0; i < 2; ++i) {
        const uint64_t e[4] = {static_cast<uint64_t>(d), static_cast<uint64_t>(page_size), static_cast<uint64_t>(Hk),
                               static_cast<uint64_t>(pages)};
        const uint64_t b[3] = {static_cast<uint64_t>(kvs[i][2]) * 2, static_cast<uint64_t>(kvs[i][1]) * 2,
                               static_cast<uint64_t>(kvs[i][0]) * 2};
        const uint32_t box[4] = {64, static_cast<uint32_t>(p.box), 1, 1};
        if ((st = encode_bf16_map(&maps[1 + i], kv[i], 4, e, b, box)) != ATTN_OK) return st;
        maps[3 + i] = maps[1 + i];  // not used
    }
    if ((st = encode_q(&maps[0], Q, p, d, R, T, qs[0], qs[1], qs[2])) != ATTN_OK) return st;
    return run<true>(*dev, maps, p, d, scale, workspace, stream);
}
