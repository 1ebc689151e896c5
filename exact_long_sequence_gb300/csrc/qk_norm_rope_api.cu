// C ABI of the query / key preparation (head norm and rotary positions) and
// its gradient: argument checks, how a token's heads are dealt to warps, launches.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/exact_attn.h"
#include "api_common.h"
#include "qk_norm_rope_kernels.cuh"

namespace elsattn {
namespace {

// Sizes, alignment and the axis ranges, shared by both directions.
int fill_params(ReadyParams& p, const int32_t* positions, int64_t pos_axis, int64_t pos_batch, const double* inv_freq,
                const int* sections, int num_sections, int B, int Hq, int Hk, int N, int d, float eps) {
    if (!positions || !inv_freq || !sections) return ATTN_ERR_INVALID_ARG;
    if (B < 1 || Hq < 1 || Hk < 1 || N < 1) return ATTN_ERR_INVALID_ARG;
    if (static_cast<long long>(B) * N >= kRoundedSizeLimit || static_cast<long long>(B) * N * Hq >= kRoundedSizeLimit ||
        static_cast<long long>(B) * N * Hk >= kRoundedSizeLimit)
        return ATTN_ERR_INVALID_ARG;
    if (!(std::isfinite(eps) && eps >= 0.f)) return ATTN_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    if (num_sections < 1 || num_sections > kReadyMaxAxes) return ATTN_ERR_INVALID_ARG;
    int pairs = 0;
    for (int a = 0; a < kReadyMaxAxes; ++a) {
        if (a < num_sections) {
            if (sections[a] < 1 || sections[a] > d) return ATTN_ERR_INVALID_ARG;
            pairs += sections[a];
        }
        p.axis_end[a] = a + 1 < num_sections ? pairs : d;  // the last axis has the rest
    }
    if (2 * pairs > d) return ATTN_ERR_INVALID_ARG;
    if (pairs % 8 != 0) return ATTN_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(positions) & 3u) != 0 || (reinterpret_cast<uintptr_t>(inv_freq) & 7u) != 0)
        return ATTN_ERR_MISALIGNED;
    p.pos = positions;
    p.pos_axis = pos_axis;
    p.pos_batch = pos_batch;
    p.inv_freq = inv_freq;
    p.rot = 2 * pairs;
    p.N.set(N);
    p.tokens = static_cast<uint32_t>(B) * static_cast<uint32_t>(N);
    p.eps = eps;
    const int group = 32 / (d / 16);
    p.t[0].H = Hq;
    p.t[1].H = Hk;
    // Several tokens side by side in a warp step, for tensors with few heads.
    // That walk costs about a fifth more per step (32768 tokens of 32 + 8 heads
    // of 128, backward: 191 us against 163 us) and saves steps where a tensor's
    // heads fill less than a step (65536 tokens of 1 + 1 heads of 64,
    // backward: 33 us against 96 us).
    double one = 0, several = 0;
    int hp[2], tp[2];
    for (int i = 0; i < 2; ++i) {
        ReadyTensor& t = p.t[i];
        t.steps = (t.H + group - 1) / group;
        for (hp[i] = 1; hp[i] < t.H && hp[i] < group;) hp[i] *= 2;
        tp[i] = group / hp[i];
        one += t.steps + 1;
        several += static_cast<double>(t.steps) / tp[i] + 1;
    }
    p.multi = 1.2 * several < one;
    for (int i = 0; i < 2; ++i) {
        p.t[i].hp = p.multi ? hp[i] : group;
        p.t[i].tp = p.multi ? tp[i] : 1;
    }
    return ATTN_OK;
}

// Strides of a [B, H, N, d] view (nullptr: contiguous), in elements.  Rows are
// moved in 16-byte vectors.  A written tensor may not repeat rows.
int take_strides(int64_t (&out)[3], const int64_t* s, int B, int H, int N, int d, bool written) {
    const int64_t dense[3] = {static_cast<int64_t>(H) * N * d, static_cast<int64_t>(N) * d, d};
    const int dims[3] = {B, H, N};
    for (int i = 0; i < 3; ++i) {
        out[i] = s ? s[i] : dense[i];
        if (dims[i] == 1) out[i] = 0;  // never stepped
        else if (out[i] % 8 != 0) return ATTN_ERR_MISALIGNED;
        else if (written && out[i] == 0) return ATTN_ERR_INVALID_ARG;
    }
    return ATTN_OK;
}

// How the work is dealt.  A warp works on one tensor: the CTAs are split
// between Q and K by their share of the steps, a step's angles counting as
// one step more (for each of its tokens).  A unit is a whole token once there are enough of them to
// give the tensor's warps one each; below that a token's heads are dealt to
// more warps.  Returns the grid.
unsigned deal_units(ReadyParams& p, int num_sms, int per_sm, int cta_warps) {
    const int64_t most = static_cast<int64_t>(num_sms) * per_sm;
    const double cost_q = static_cast<double>(p.t[0].steps) / p.t[0].tp + 1, cost_k = static_cast<double>(p.t[1].steps) / p.t[1].tp + 1;
    int64_t ctas[2];
    ctas[0] = static_cast<int64_t>(std::lround(most * cost_q / (cost_q + cost_k)));
    if (ctas[0] < 1) ctas[0] = 1;
    if (ctas[0] > most - 1) ctas[0] = most - 1;
    ctas[1] = most - ctas[0];
    for (int t = 0; t < 2; ++t) {
        ReadyTensor& r = p.t[t];
        const int64_t warps = ctas[t] * cta_warps;
        const uint32_t groups = (p.tokens + r.tp - 1) / r.tp;
        const int64_t want = (static_cast<int64_t>(r.steps) * groups + warps - 1) / warps;
        r.steps_per_unit = static_cast<int>(want < 1 ? 1 : want > r.steps ? r.steps : want);
        const int per_token = (r.steps + r.steps_per_unit - 1) / r.steps_per_unit;
        r.units_per_token.set(per_token);
        // more than one a token only while there are fewer units than warps: below 2^31
        r.units = groups * static_cast<uint32_t>(per_token);
        const int64_t need = (static_cast<int64_t>(r.units) + cta_warps - 1) / cta_warps;
        if (need < ctas[t]) ctas[t] = need;
        r.part = nullptr;
    }
    p.first_k = static_cast<int>(ctas[0]);
    return static_cast<unsigned>(ctas[0] + ctas[1]);
}

// By <d == 128><interleaved><several tokens a step>.
using ReadyKernel = void (*)(ReadyParams);
#define ELS_READY_KERNELS(K, U)                                                                         \
    {K<64, false, U, false>, K<64, false, U, true>, K<64, true, U, false>, K<64, true, U, true>,        \
     K<128, false, U, false>, K<128, false, U, true>, K<128, true, U, false>, K<128, true, U, true>}
const ReadyKernel kFwdKernels[8] = ELS_READY_KERNELS(qk_norm_rope_kernel, kFwdSlots);
const ReadyKernel kBwdKernels[8] = ELS_READY_KERNELS(qk_norm_rope_bwd_kernel, kBwdSlots);
#undef ELS_READY_KERNELS

constexpr int kFwdSmem = kFwdWarps * ReadyRing<128, 2, kFwdSlots, false>::kBytes;
constexpr int kBwdSmem = kBwdWarps * ReadyRing<128, 4, kBwdSlots, false>::kBytes;

// Once per device and kernel (a second call that races with the first sets the same limit again).
int allow_smem(bool& done, ReadyKernel kernel, int bytes) {
    if (done) return ATTN_OK;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return cuda_fail(e);
    done = true;
    return ATTN_OK;
}

int launched() {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

}  // namespace
}  // namespace elsattn

using namespace elsattn;

extern "C" int attn_qk_norm_rope(const void* Q, const int64_t* q_strides, const void* K, const int64_t* k_strides,
                                 const void* q_weight, const void* k_weight, const int32_t* positions,
                                 int64_t pos_axis_stride, int64_t pos_batch_stride, const double* inv_freq,
                                 const int* sections, int num_sections, void* Qout, const int64_t* qo_strides,
                                 void* Kout, const int64_t* ko_strides, int B, int Hq, int Hk, int N, int d, float eps,
                                 int interleaved, cudaStream_t stream) {
    if (!Q || !K || !Qout || !Kout) return ATTN_ERR_INVALID_ARG;
    ReadyParams p;
    int st = fill_params(p, positions, pos_axis_stride, pos_batch_stride, inv_freq, sections, num_sections, B, Hq, Hk,
                         N, d, eps);
    if (st != ATTN_OK) return st;
    const void* in[2] = {Q, K};
    void* out[2] = {Qout, Kout};
    const void* w[2] = {q_weight, k_weight};
    const int64_t *xs[2] = {q_strides, k_strides}, *ys[2] = {qo_strides, ko_strides};
    for (int t = 0; t < 2; ++t) {
        ReadyTensor& r = p.t[t];
        if (!aligned16(in[t]) || !aligned16(out[t]) || !aligned16(w[t])) return ATTN_ERR_MISALIGNED;
        if ((st = take_strides(r.xs, xs[t], B, r.H, N, d, false)) != ATTN_OK ||
            (st = take_strides(r.ys, ys[t], B, r.H, N, d, true)) != ATTN_OK)
            return st;
        r.x = static_cast<const __nv_bfloat16*>(in[t]);
        r.g = nullptr;
        r.y = static_cast<__nv_bfloat16*>(out[t]);
        r.w = static_cast<const __nv_bfloat16*>(w[t]);
    }
    DeviceState* dev = nullptr;
    if ((st = device_state(&dev)) != ATTN_OK) return st;
    const unsigned grid = deal_units(p, dev->num_sms, kFwdCtasPerSm, kFwdWarps);
    const int variant = (d == 128 ? 4 : 0) + (interleaved ? 2 : 0) + (p.multi ? 1 : 0);
    const ReadyKernel kernel = kFwdKernels[variant];
    if ((st = allow_smem(dev->ready_configured[0][variant], kernel, kFwdSmem)) != ATTN_OK) return st;
    kernel<<<grid, kFwdWarps * 32, kFwdSmem, stream>>>(p);
    return launched();
}

extern "C" size_t attn_qk_norm_rope_bwd_workspace_bytes(int d) {
    if (d != 64 && d != 128) return 0;
    DeviceState* dev = nullptr;
    if (device_state(&dev) != ATTN_OK) return 0;
    return static_cast<size_t>(dev->num_sms) * kBwdCtasPerSm * d * sizeof(float);
}

extern "C" int attn_qk_norm_rope_bwd(const void* dQout, const int64_t* dqo_strides, const void* dKout,
                                     const int64_t* dko_strides, const void* Q, const int64_t* q_strides, const void* K,
                                     const int64_t* k_strides, const void* q_weight, const void* k_weight,
                                     const int32_t* positions, int64_t pos_axis_stride, int64_t pos_batch_stride,
                                     const double* inv_freq, const int* sections, int num_sections, void* dQ,
                                     const int64_t* dq_strides, void* dK, const int64_t* dk_strides, float* dq_weight,
                                     float* dk_weight, int B, int Hq, int Hk, int N, int d, float eps, int interleaved,
                                     void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!dQout || !dKout || !dQ || !dK) return ATTN_ERR_INVALID_ARG;
    ReadyParams p;
    int st = fill_params(p, positions, pos_axis_stride, pos_batch_stride, inv_freq, sections, num_sections, B, Hq, Hk,
                         N, d, eps);
    if (st != ATTN_OK) return st;
    const void *up[2] = {dQout, dKout}, *in[2] = {Q, K}, *w[2] = {q_weight, k_weight};
    void* out[2] = {dQ, dK};
    float* dw[2] = {dq_weight, dk_weight};
    const int64_t *gs[2] = {dqo_strides, dko_strides}, *xs[2] = {q_strides, k_strides}, *ys[2] = {dq_strides, dk_strides};
    bool any_norm = false;
    for (int t = 0; t < 2; ++t) {
        ReadyTensor& r = p.t[t];
        // a norm has an input to differentiate at and a weight gradient to write; without one there is neither
        if ((w[t] != nullptr) != (dw[t] != nullptr) || (w[t] && !in[t])) return ATTN_ERR_INVALID_ARG;
        if (!aligned16(up[t]) || !aligned16(out[t]) || !aligned16(w[t]) || (w[t] && !aligned16(in[t])))
            return ATTN_ERR_MISALIGNED;
        if ((reinterpret_cast<uintptr_t>(dw[t]) & 3u) != 0) return ATTN_ERR_MISALIGNED;
        if ((st = take_strides(r.gs, gs[t], B, r.H, N, d, false)) != ATTN_OK ||
            (st = take_strides(r.ys, ys[t], B, r.H, N, d, true)) != ATTN_OK ||
            (w[t] && (st = take_strides(r.xs, xs[t], B, r.H, N, d, false)) != ATTN_OK))
            return st;
        r.g = static_cast<const __nv_bfloat16*>(up[t]);
        r.x = static_cast<const __nv_bfloat16*>(in[t]);
        r.y = static_cast<__nv_bfloat16*>(out[t]);
        r.w = static_cast<const __nv_bfloat16*>(w[t]);
        any_norm = any_norm || w[t];
    }
    if (any_norm) {
        if (!workspace) return ATTN_ERR_INVALID_ARG;
        if (!aligned16(workspace)) return ATTN_ERR_MISALIGNED;
    }
    DeviceState* dev = nullptr;
    if ((st = device_state(&dev)) != ATTN_OK) return st;
    if (any_norm && workspace_bytes < attn_qk_norm_rope_bwd_workspace_bytes(d)) return ATTN_ERR_INVALID_ARG;
    const unsigned grid = deal_units(p, dev->num_sms, kBwdCtasPerSm, kBwdWarps);
    ReadyDw sums;
    const int first[2] = {0, p.first_k}, rows[2] = {p.first_k, static_cast<int>(grid) - p.first_k};
    for (int t = 0; t < 2; ++t) {
        p.t[t].part = w[t] ? static_cast<float*>(workspace) + static_cast<size_t>(first[t]) * d : nullptr;
        sums.part[t] = p.t[t].part;
        sums.rows[t] = rows[t];
        sums.dw[t] = dw[t];
    }
    const int variant = (d == 128 ? 4 : 0) + (interleaved ? 2 : 0) + (p.multi ? 1 : 0);
    const ReadyKernel grad = kBwdKernels[variant];
    if ((st = allow_smem(dev->ready_configured[1][variant], grad, kBwdSmem)) != ATTN_OK) return st;
    grad<<<grid, kBwdWarps * 32, kBwdSmem, stream>>>(p);
    if ((st = launched()) != ATTN_OK || !any_norm) return st;
    // its CTAs may start as the gradient kernel's retire, and wait in-kernel for its completion
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(d / 32), 2);
    cfg.blockDim = dim3(1024);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const auto kernel = d == 64 ? qk_norm_rope_dw_kernel<64> : qk_norm_rope_dw_kernel<128>;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, sums);
    return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}
