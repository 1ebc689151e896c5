// C ABI of the gradients of attention over packed sequences: argument checks,
// the cut of the work, TMA descriptors, launches.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/exact_attn.h"
#include "api_common.h"
#include "attn_packed_bwd_kernel.cuh"

namespace elsattn {
namespace {

// Q, dO and the sums of dQ that the CTAs work on at a time: the line has a stretch a CTA for each so many bytes, up to
// kBwdMostTurns.  A turn's bytes stay in L2; each costs its stretches' pieces (40 MB at d = 128).  32 texts of 2048 tokens, 32
// heads of 8, with 4, 8, 12 and 15 turns: 4347, 3832, 3617 and 3606 us; 4 documents of 16384 with 4 and 15: 23.7 and 20.9 ms.
// Between 150 and 200 MB a turn it is about even: the fourth turn of 24 texts of 10 to 2501 tokens, 24 heads of 4, costs
// 757 us for 744, and documents of up to 16384 tokens, 16 heads of 8, read 2.7 GB in place of 6.5 in the same time.
constexpr double kBwdTurnBytes = 150e6;
constexpr int kBwdMostTurns = 32;

int check(int R, int Nq, int Nk, int Hq, int Hk, int d) {
    if (R < 1 || Nq < 1 || Nk < 1 || Hq < 1 || Hk < 1 || Hq % Hk != 0) return ATTN_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    if (Hq / Hk > kPkMostGroup) return ATTN_ERR_UNSUPPORTED;
    if (static_cast<long long>(Hq) * Nq >= kRoundedSizeLimit || static_cast<long long>(Hk) * Nk >= kRoundedSizeLimit ||
        R >= kRoundedSizeLimit)
        return ATTN_ERR_INVALID_ARG;
    return ATTN_OK;
}

void lay_out(PackedBwdParams& p, int Nq, int Hq, int Hk, int d, int num_sms) {
    p.Hk = Hk;
    p.G = Hq / Hk;
    p.block_tokens = kBq / p.G;
    p.qrows = p.block_tokens * p.G;
    int turns = static_cast<int>(std::fmin(std::ceil(8.0 * Nq * Hq * d / kBwdTurnBytes), kBwdMostTurns));
    if (turns < 1) turns = 1;
    p.stretches = num_sms * turns;
    // Up to eight blocks of tokens no unit is cut: each is left whole in the stretch where it starts (it may be nearly two of the
    // shortest stretches long, with its own 7 blocks), and the workspace holds no pieces.
    p.whole = Nq <= kKeyLineLeast * p.block_tokens;
}

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// Workspace: cuts and whether the offsets fall, D of every row, dQ's sums, pieces of dV and dK.
struct Space {
    size_t dvec, dq, part, bytes;
    Space(const PackedBwdParams& p, int Nq, int d) {
        const size_t rows = static_cast<size_t>(p.Hk) * p.G * Nq;
        dvec = align256(p.stretches * sizeof(PackedBwdCut) + sizeof(int));
        dq = dvec + align256(rows * sizeof(float));
        part = dq + rows * d * sizeof(float);
        bytes = part + (p.whole ? 0 : 2 * static_cast<size_t>(p.stretches) * kBc * 2 * d * sizeof(float));
    }
};

template <int D>
int launch(DeviceState& dev, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mdo,
           const PackedBwdParams& p, const PackedRowParams& rows, float* dvec, cudaStream_t stream) {
    auto kernel = attn_packed_bwd_kernel<D>;
    constexpr int smem = PackedBwdLayout<D>::kSmem;
    bool& configured = dev.packed_bwd_smem_configured[D == 128];
    cudaError_t e;
    if (!configured) {
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
            return cuda_fail(e);
        configured = true;
    }
    const int64_t threads = static_cast<int64_t>(rows.Hq) * rows.Nq * (D / 8);
    const unsigned blocks = static_cast<unsigned>((threads + 255) / 256);
    // The first launch is a plain one: a programmatic dependent waits for the grid before it only, and where the caller's
    // own grid is one that does not wait for those before, these could still run.
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(256);
    if ((e = cudaLaunchKernelEx(&cfg, attn_packed_bwd_prep_kernel<D>, rows, dvec, p.dq_acc, p.scale)) != cudaSuccess)
        return cuda_fail(e);
    // The other two each depend on the one before them, and wait for it once they are set up.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(dev.num_sms));
    cfg.blockDim = dim3(kBwdThreads);
    cfg.dynamicSmemBytes = smem;
    if ((e = cudaLaunchKernelEx(&cfg, kernel, mq, mk, mv, mdo, p)) != cudaSuccess) return cuda_fail(e);
    cfg.dynamicSmemBytes = 0;
    cfg.gridDim = dim3((blocks + 1) / 2 + (p.whole ? 0u : static_cast<unsigned>(p.stretches) * kPkbCutCtas));
    cfg.blockDim = dim3(256);
    if ((e = cudaLaunchKernelEx(&cfg, attn_packed_bwd_post_kernel<D>, p, rows)) != cudaSuccess) return cuda_fail(e);
    return ATTN_OK;
}

}  // namespace
}  // namespace elsattn

using namespace elsattn;

extern "C" size_t attn_bwd_packed_workspace_bytes(int R, int Nq, int Nk, int Hq, int Hk, int d) {
    if (check(R, Nq, Nk, Hq, Hk, d) != ATTN_OK) return 0;
    DeviceState* dev = nullptr;
    if (device_state(&dev) != ATTN_OK) return 0;
    PackedBwdParams p{};
    lay_out(p, Nq, Hq, Hk, d, dev->num_sms);
    return Space(p, Nq, d).bytes;
}

extern "C" int attn_bwd_packed(const void* Q, const int64_t* q_strides, const void* K, const int64_t* k_strides, const void* V,
                               const int64_t* v_strides, const void* O, const int64_t* o_strides, const float* LSE,
                               const void* dO, const int64_t* do_strides, const int32_t* q_starts, const int32_t* k_starts,
                               void* dQ, const int64_t* dq_strides, void* dK, const int64_t* dk_strides, void* dV,
                               const int64_t* dv_strides, int R, int Nq, int Nk, int Hq, int Hk, int d, int causal, float scale,
                               void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    int st = check(R, Nq, Nk, Hq, Hk, d);
    if (st != ATTN_OK) return st;
    const void* tensors[8] = {Q, K, V, O, dO, dQ, dK, dV};
    for (const void* t : tensors)
        if (!t) return ATTN_ERR_INVALID_ARG;
    if (!LSE || !q_starts || !k_starts || !workspace || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
    for (const void* t : tensors)
        if (!aligned16(t)) return ATTN_ERR_MISALIGNED;
    if (!aligned16(workspace) ||
        ((reinterpret_cast<uintptr_t>(LSE) | reinterpret_cast<uintptr_t>(q_starts) | reinterpret_cast<uintptr_t>(k_starts)) & 3u) != 0)
        return ATTN_ERR_MISALIGNED;
    PackedBwdParams p{};
    PackedRowParams rows{};
    int64_t qs[2], ks[2], vs[2];
    const int64_t q_dims[2] = {Hq, Nq}, k_dims[2] = {Hk, Nk};
    if ((st = take_view(qs, q_strides, q_dims, d)) != ATTN_OK || (st = take_view(ks, k_strides, k_dims, d)) != ATTN_OK ||
        (st = take_view(vs, v_strides, k_dims, d)) != ATTN_OK || (st = take_view(rows.os, o_strides, q_dims, d)) != ATTN_OK ||
        (st = take_view(rows.dos, do_strides, q_dims, d)) != ATTN_OK ||
        (st = take_view(rows.dqs, dq_strides, q_dims, d)) != ATTN_OK ||
        (st = take_view(p.dks, dk_strides, k_dims, d)) != ATTN_OK || (st = take_view(p.dvs, dv_strides, k_dims, d)) != ATTN_OK)
        return st;
    DeviceState* dev = nullptr;
    if ((st = device_state(&dev)) != ATTN_OK) return st;
    lay_out(p, Nq, Hq, Hk, d, dev->num_sms);
    const Space space(p, Nq, d);
    if (workspace_bytes < space.bytes) return ATTN_ERR_INVALID_ARG;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    float* dvec = reinterpret_cast<float*>(ws + space.dvec);
    p.cuts = reinterpret_cast<PackedBwdCut*>(ws);
    p.falls = reinterpret_cast<int*>(p.cuts + p.stretches);
    p.dvec = dvec;
    p.dq_acc = reinterpret_cast<float*>(ws + space.dq);
    p.part = reinterpret_cast<float*>(ws + space.part);
    p.q_starts = q_starts;
    p.k_starts = k_starts;
    p.lse = LSE;
    p.dk = static_cast<__nv_bfloat16*>(dK);
    p.dv = static_cast<__nv_bfloat16*>(dV);
    p.R = R;
    p.Nq = Nq;
    p.Nk = Nk;
    p.causal = causal != 0;
    p.error_word = dev->error_word;
    p.scale = scale;
    p.scale_log2 = scale * 1.4426950408889634f;
    rows.o = static_cast<const __nv_bfloat16*>(O);
    rows.dout = static_cast<const __nv_bfloat16*>(dO);
    rows.dq = static_cast<__nv_bfloat16*>(dQ);
    rows.Hq = Hq;
    rows.G = p.G;
    rows.Nq = Nq;
    CUtensorMap mq, mk, mv, mdo;
    auto q_map = [&](CUtensorMap* map, const void* t, const int64_t* s) {
        const uint64_t e[4] = {static_cast<uint64_t>(d), static_cast<uint64_t>(p.G), static_cast<uint64_t>(Hk), static_cast<uint64_t>(Nq)};
        const uint64_t b[3] = {static_cast<uint64_t>(s[0]) * 2, static_cast<uint64_t>(s[0]) * p.G * 2, static_cast<uint64_t>(s[1]) * 2};
        const uint32_t box[4] = {64, static_cast<uint32_t>(p.G), 1, static_cast<uint32_t>(p.block_tokens)};
        return encode_bf16_map(map, t, 4, e, b, box);
    };
    auto k_map = [&](CUtensorMap* map, const void* t, const int64_t* s) {
        const uint64_t e[3] = {static_cast<uint64_t>(d), static_cast<uint64_t>(Nk), static_cast<uint64_t>(Hk)};
        const uint64_t b[2] = {static_cast<uint64_t>(s[1]) * 2, static_cast<uint64_t>(s[0]) * 2};
        const uint32_t box[3] = {64, kBc, 1};
        return encode_bf16_map(map, t, 3, e, b, box);
    };
    if ((st = q_map(&mq, Q, qs)) != ATTN_OK || (st = q_map(&mdo, dO, rows.dos)) != ATTN_OK ||
        (st = k_map(&mk, K, ks)) != ATTN_OK || (st = k_map(&mv, V, vs)) != ATTN_OK)
        return st;
    p.timeout_ns = kDefaultTimeoutNs;
    if (const uint64_t t = take_armed_timeout()) {  // (test hook)
        p.timeout_ns = t;
        p.withhold_first_block = 1u;
    }
    return d == 64 ? launch<64>(*dev, mq, mk, mv, mdo, p, rows, dvec, stream)
                   : launch<128>(*dev, mq, mk, mv, mdo, p, rows, dvec, stream);
}
