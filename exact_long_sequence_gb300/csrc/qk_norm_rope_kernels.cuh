// Queries and keys made ready for attention on sm_103a, and the gradient of
// that step: RMS normalisation of each head's row and the rotation by the
// token's position, in one pass over Q and K.
//
// Forward, per row x of d elements (one token, one head), in fp32:
//     y = x * rsqrt(mean(x^2) + eps) * w            (w = nullptr: y = x)
//     (y_a, y_b) -> (y_a cos t - y_b sin t, y_b cos t + y_a sin t)  for each pair,
// where pair i turns by t = position[axis(i)] * inv_freq[i]; elements past the
// rotated ones keep y.  Rounded once, to bf16, at the end.
// Backward, for an upstream gradient g of the output: u = R^T g (the turn by
// -t), h = x r with r = rsqrt(mean(x^2) + eps),
//     dx = r (u w - h mean(u w h)),   dw = sum over rows of u h.
//
// Both are bound by HBM: a row is read once and written once, nothing else of
// its size moves.  A row of d elements is held by d / 16 lanes, 16 elements
// each as two 16-byte vectors placed so that both members of a pair are in one
// lane; a warp holds 32 / (d / 16) rows (heads) of one token at a time, so the
// token's sines and cosines are computed once per warp, each lane evaluating
// the share of pairs that its row group would otherwise repeat, and are passed
// around by shuffles.
//
// Angles: a position times a frequency loses its fraction of a turn in fp32
// (position 10^6 at frequency 1 is off by 0.06 rad).  Here the frequency is
// held as a 64-bit fixed-point fraction of a turn, F = inv_freq / (2 pi) mod 1
// times 2^64, so that position * F mod 2^64 is the angle mod one turn, exact but
// for F's own rounding (2^-53 of a turn times the position): one integer product.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "rowwise_kernels.cuh"
#include "sm103_ptx.cuh"

namespace elsattn {

constexpr int kReadyMaxAxes = 4;
constexpr int kReadyWarps = 8;  // per CTA

struct ReadyTensor {
    const __nv_bfloat16* x;   // input rows (backward: the forward's input; unused without a norm)
    const __nv_bfloat16* g;   // backward: gradient of the output rows
    __nv_bfloat16* y;         // output rows (backward: gradient of the input rows)
    const __nv_bfloat16* w;   // [d] norm weight, or nullptr: no norm
    int64_t xs[3], gs[3], ys[3];  // strides in elements: batch, head, token
    int H;
    int steps;                // warp steps per token: ceil(H / rows per warp)
};

struct ReadyParams {
    ReadyTensor t[2];         // Q, K
    const int32_t* pos;       // position of token n of batch b on axis a: pos[a * pos_axis + b * pos_batch + n]
    int64_t pos_axis, pos_batch;
    const double* inv_freq;   // [rot / 2]
    int axis_end[kReadyMaxAxes];  // pairs [axis_end[a - 1], axis_end[a]) turn by axis a
    int rot;                  // rotated elements of a row
    int N;
    uint32_t tokens;          // B * N
    float eps;
    int steps_per_unit;       // a work unit: so many steps of one token
    int units_per_token;
    uint32_t units;
    float* part;              // backward: [gridDim.x][2][d] fp32 partial sums of dw
};

// The pair that lane `c` of a row group holds as its k-th (0..7), and whether
// it is rotated.  Halves: lane c holds elements 8c.. and rot/2 + 8c.. (the
// pairs 8c .. 8c + 7); lanes past them hold 16 neighbouring unrotated elements.
// Neighbours: lane c holds elements 8c.. and d/2 + 8c.., four pairs each.
template <int D, bool INTER>
struct ReadyLane {
    int a0, b0;       // element offsets of the two vectors
    bool rot_a, rot_b;
    __device__ __forceinline__ ReadyLane(int c, int rot) {
        if (INTER) {
            a0 = 8 * c;
            b0 = D / 2 + 8 * c;
            rot_a = a0 < rot;
            rot_b = b0 < rot;
        } else {
            const int half = rot >> 1;
            rot_a = rot_b = 8 * c < half;
            a0 = rot_a ? 8 * c : rot + 2 * (8 * c - half);
            b0 = rot_a ? half + 8 * c : a0 + 8;
        }
    }
    __device__ static __forceinline__ int pair(int c, int k) {
        return INTER ? (k < 4 ? 4 * c + k : D / 4 + 4 * c + (k - 4)) : 8 * c + k;
    }
};

// A frequency as a fraction of a turn in 64-bit fixed point.
__device__ __forceinline__ uint64_t turn_fraction(double inv_freq) {
    double f = inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
    f -= floor(f);
    if (!(f < 1.0)) return 0;  // rounded up to a whole turn (or not finite)
    const double hi = floor(f * 4294967296.0);  // exact: a power of two times f
    const double lo = (f * 4294967296.0 - hi) * 4294967296.0;
    return (static_cast<uint64_t>(static_cast<uint32_t>(hi)) << 32) | static_cast<uint64_t>(lo);
}

// Cosines and sines of the pairs this lane's elements belong to, for one
// token.  The rows of a warp share the token, so of the 8 pairs that the lanes
// with the same c need, each of the kGroups row groups evaluates 8 / kGroups.
template <int D>
struct ReadyAngles {
    static constexpr int kLanes = D / 16;        // lanes per row
    static constexpr int kGroups = 32 / kLanes;  // rows per warp step
    static constexpr int kOwn = 8 / kGroups;     // pairs evaluated per lane
    uint64_t f[kOwn];
    int axis[kOwn];

    template <bool INTER>
    __device__ __forceinline__ void init(const ReadyParams& p, int lane) {
        const int c = lane % kLanes, g = lane / kLanes;
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            const int i = ReadyLane<D, INTER>::pair(c, g * kOwn + k);
            f[k] = 0;
            axis[k] = 0;
            if (i < (p.rot >> 1)) {
                f[k] = turn_fraction(p.inv_freq[i]);
#pragma unroll
                for (int a = 0; a < kReadyMaxAxes - 1; ++a) axis[k] += i >= p.axis_end[a] ? 1 : 0;
            }
        }
    }
    // The positions of a token, one per evaluated pair (issued early).
    __device__ __forceinline__ void load(const ReadyParams& p, int b, int n, int (&pos)[kOwn]) const {
#pragma unroll
        for (int k = 0; k < kOwn; ++k)
            pos[k] = p.pos[axis[k] * p.pos_axis + b * p.pos_batch + n];
    }
    __device__ __forceinline__ void eval(const int (&pos)[kOwn], int lane, float (&cs)[8], float (&sn)[8]) const {
        float c0[kOwn], s0[kOwn];
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            const uint64_t turn = f[k] * static_cast<uint64_t>(static_cast<int64_t>(pos[k]));
            // the top 32 bits as a signed fraction of a turn, [-1/2, 1/2); in units of pi: [-1, 1)
            const float x = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f;
            sincospif(x, &s0[k], &c0[k]);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int src = (k / kOwn) * kLanes + lane % kLanes;
            cs[k] = __shfl_sync(0xffffffffu, c0[k % kOwn], src);
            sn[k] = __shfl_sync(0xffffffffu, s0[k % kOwn], src);
        }
    }
};

// Sum over the lanes of a row.
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Turn the lane's pairs by the angles (SIGN = 1) or back (SIGN = -1).  a, b:
// the two vectors.
template <bool INTER, int SIGN>
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], bool rot_a, bool rot_b, const float (&cs)[8],
                                     const float (&sn)[8]) {
    if (INTER) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (rot_a) {
                const float x = a[2 * k], y = a[2 * k + 1], s = SIGN * sn[k];
                a[2 * k] = x * cs[k] - y * s;
                a[2 * k + 1] = y * cs[k] + x * s;
            }
            if (rot_b) {
                const float x = b[2 * k], y = b[2 * k + 1], s = SIGN * sn[4 + k];
                b[2 * k] = x * cs[4 + k] - y * s;
                b[2 * k + 1] = y * cs[4 + k] + x * s;
            }
        }
    } else if (rot_a) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float x = a[k], y = b[k], s = SIGN * sn[k];
            a[k] = x * cs[k] - y * s;
            b[k] = y * cs[k] + x * s;
        }
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ uint4 ld16(const __nv_bfloat16* p) { return *reinterpret_cast<const uint4*>(p); }

// U: steps whose loads are in flight together.
template <int D, bool INTER, int U>
__global__ void __launch_bounds__(kReadyWarps * 32) qk_norm_rope_kernel(const __grid_constant__ ReadyParams p) {
    using A = ReadyAngles<D>;
    const int lane = threadIdx.x & 31;
    const int c = lane % A::kLanes, g = lane / A::kLanes;
    const ReadyLane<D, INTER> at(c, p.rot);
    A angles;
    angles.template init<INTER>(p, lane);
    // both tensors' weights for this lane's elements, as bf16
    uint4 w[2][2] = {};
#pragma unroll
    for (int t = 0; t < 2; ++t)
        if (p.t[t].w) {
            w[t][0] = ld16(p.t[t].w + at.a0);
            w[t][1] = ld16(p.t[t].w + at.b0);
        }
    const int total = p.t[0].steps + p.t[1].steps;
    const uint32_t warps = gridDim.x * kReadyWarps;
    for (uint32_t u = blockIdx.x * kReadyWarps + (threadIdx.x >> 5); u < p.units; u += warps) {
        const uint32_t token = u / p.units_per_token;
        const int s0 = static_cast<int>(u - token * p.units_per_token) * p.steps_per_unit;
        const int s1 = min(total, s0 + p.steps_per_unit);
        const int b = static_cast<int>(token / static_cast<uint32_t>(p.N));
        const int n = static_cast<int>(token - static_cast<uint32_t>(b) * p.N);
        int pos[A::kOwn];
        angles.load(p, b, n, pos);
        float cs[8], sn[8];
        for (int s = s0; s < s1; s += U) {
            uint4 va[U], vb[U];
            bool on[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int t = s + j >= p.t[0].steps ? 1 : 0;
                const ReadyTensor& rt = p.t[t];
                const int h = (s + j - (t ? p.t[0].steps : 0)) * A::kGroups + g;
                on[j] = s + j < s1 && h < rt.H;
                va[j] = vb[j] = make_uint4(0, 0, 0, 0);
                if (on[j]) {
                    const __nv_bfloat16* row = rt.x + b * rt.xs[0] + h * rt.xs[1] + n * rt.xs[2];
                    va[j] = ld_stream(reinterpret_cast<const uint4*>(row + at.a0));
                    vb[j] = ld_stream(reinterpret_cast<const uint4*>(row + at.b0));
                }
            }
            if (s == s0) angles.eval(pos, lane, cs, sn);
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (s + j >= s1) break;
                const int t = s + j >= p.t[0].steps ? 1 : 0;
                const ReadyTensor& rt = p.t[t];
                const int h = (s + j - (t ? p.t[0].steps : 0)) * A::kGroups + g;
                float a[8], bb[8];
                bf16x8_to_float(va[j], a);
                bf16x8_to_float(vb[j], bb);
                if (rt.w) {
                    float ss = 0.f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) ss = fmaf(a[k], a[k], fmaf(bb[k], bb[k], ss));
                    const float r = rsqrtf(row_sum<A::kLanes>(ss) * (1.0f / D) + p.eps);
                    float wa[8], wb[8];
                    bf16x8_to_float(t ? w[1][0] : w[0][0], wa);
                    bf16x8_to_float(t ? w[1][1] : w[0][1], wb);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        a[k] *= r * wa[k];
                        bb[k] *= r * wb[k];
                    }
                }
                turn<INTER, 1>(a, bb, at.rot_a, at.rot_b, cs, sn);
                if (on[j]) {
                    __nv_bfloat16* row = rt.y + b * rt.ys[0] + h * rt.ys[1] + n * rt.ys[2];
                    *reinterpret_cast<uint4*>(row + at.a0) = pack8(a);
                    *reinterpret_cast<uint4*>(row + at.b0) = pack8(bb);
                }
            }
        }
    }
}

// The gradient.  dw is summed per lane in fp32 over the warp's rows, then over
// the row groups of the warp, the warps of the CTA (both in a fixed order), and
// by qk_norm_rope_dw_kernel over the CTAs: the same inputs give the same bits.
template <int D, bool INTER, int U>
__global__ void __launch_bounds__(kReadyWarps * 32, 2) qk_norm_rope_bwd_kernel(const __grid_constant__ ReadyParams p) {
    using A = ReadyAngles<D>;
    __shared__ float s_dw[kReadyWarps][2][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = lane % A::kLanes, g = lane / A::kLanes;
    const ReadyLane<D, INTER> at(c, p.rot);
    A angles;
    angles.template init<INTER>(p, lane);
    uint4 w[2][2] = {};
#pragma unroll
    for (int t = 0; t < 2; ++t)
        if (p.t[t].w) {
            w[t][0] = ld16(p.t[t].w + at.a0);
            w[t][1] = ld16(p.t[t].w + at.b0);
        }
    float acc[2][16];
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[0][k] = acc[1][k] = 0.f;
    const int total = p.t[0].steps + p.t[1].steps;
    const uint32_t warps = gridDim.x * kReadyWarps;
    for (uint32_t u = blockIdx.x * kReadyWarps + warp; u < p.units; u += warps) {
        const uint32_t token = u / p.units_per_token;
        const int s0 = static_cast<int>(u - token * p.units_per_token) * p.steps_per_unit;
        const int s1 = min(total, s0 + p.steps_per_unit);
        const int b = static_cast<int>(token / static_cast<uint32_t>(p.N));
        const int n = static_cast<int>(token - static_cast<uint32_t>(b) * p.N);
        int pos[A::kOwn];
        angles.load(p, b, n, pos);
        float cs[8], sn[8];
        for (int s = s0; s < s1; s += U) {
            uint4 ga[U], gb[U], xa[U], xb[U];
            bool on[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int t = s + j >= p.t[0].steps ? 1 : 0;
                const ReadyTensor& rt = p.t[t];
                const int h = (s + j - (t ? p.t[0].steps : 0)) * A::kGroups + g;
                on[j] = s + j < s1 && h < rt.H;
                ga[j] = gb[j] = xa[j] = xb[j] = make_uint4(0, 0, 0, 0);
                if (on[j]) {
                    const __nv_bfloat16* gr = rt.g + b * rt.gs[0] + h * rt.gs[1] + n * rt.gs[2];
                    ga[j] = ld_stream(reinterpret_cast<const uint4*>(gr + at.a0));
                    gb[j] = ld_stream(reinterpret_cast<const uint4*>(gr + at.b0));
                    if (rt.w) {
                        const __nv_bfloat16* xr = rt.x + b * rt.xs[0] + h * rt.xs[1] + n * rt.xs[2];
                        xa[j] = ld_stream(reinterpret_cast<const uint4*>(xr + at.a0));
                        xb[j] = ld_stream(reinterpret_cast<const uint4*>(xr + at.b0));
                    }
                }
            }
            if (s == s0) angles.eval(pos, lane, cs, sn);
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (s + j >= s1) break;
                const int t = s + j >= p.t[0].steps ? 1 : 0;
                const ReadyTensor& rt = p.t[t];
                const int h = (s + j - (t ? p.t[0].steps : 0)) * A::kGroups + g;
                float ua[8], ub[8];
                bf16x8_to_float(ga[j], ua);
                bf16x8_to_float(gb[j], ub);
                turn<INTER, -1>(ua, ub, at.rot_a, at.rot_b, cs, sn);
                if (rt.w) {
                    float ha[8], hb[8], wa[8], wb[8];
                    bf16x8_to_float(xa[j], ha);
                    bf16x8_to_float(xb[j], hb);
                    bf16x8_to_float(t ? w[1][0] : w[0][0], wa);
                    bf16x8_to_float(t ? w[1][1] : w[0][1], wb);
                    float ss = 0.f, dot = 0.f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        ss = fmaf(ha[k], ha[k], fmaf(hb[k], hb[k], ss));
                        dot = fmaf(ua[k] * wa[k], ha[k], fmaf(ub[k] * wb[k], hb[k], dot));
                    }
                    // a lane without a row adds nothing to dw, also where eps is 0
                    const float rr = rsqrtf(row_sum<A::kLanes>(ss) * (1.0f / D) + p.eps);
                    const float r = on[j] ? rr : 0.f;
                    const float m = row_sum<A::kLanes>(dot) * r * (1.0f / D);  // mean(u w h)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        ha[k] *= r;
                        hb[k] *= r;
                    }
                    if (t == 0) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            acc[0][k] = fmaf(ua[k], ha[k], acc[0][k]);
                            acc[0][8 + k] = fmaf(ub[k], hb[k], acc[0][8 + k]);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            acc[1][k] = fmaf(ua[k], ha[k], acc[1][k]);
                            acc[1][8 + k] = fmaf(ub[k], hb[k], acc[1][8 + k]);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        ua[k] = r * fmaf(-ha[k], m, ua[k] * wa[k]);
                        ub[k] = r * fmaf(-hb[k], m, ub[k] * wb[k]);
                    }
                }
                if (on[j]) {
                    __nv_bfloat16* row = rt.y + b * rt.ys[0] + h * rt.ys[1] + n * rt.ys[2];
                    *reinterpret_cast<uint4*>(row + at.a0) = pack8(ua);
                    *reinterpret_cast<uint4*>(row + at.b0) = pack8(ub);
                }
            }
        }
    }
    if (!p.part) return;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            float v = acc[t][k];
#pragma unroll
            for (int off = 16; off >= A::kLanes; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
            if (g == 0) s_dw[warp][t][(k < 8 ? at.a0 : at.b0 - 8) + k] = v;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += blockDim.x) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kReadyWarps; ++k) v += s_dw[k][i / D][i % D];
        p.part[static_cast<size_t>(blockIdx.x) * 2 * D + i] = v;
    }
}

// dw of both tensors from the CTAs' partial sums: 32 columns a CTA, the rows
// dealt to 32 warps and their sums added in a fixed order.
template <int D>
__global__ void __launch_bounds__(1024) qk_norm_rope_dw_kernel(const float* part, int rows, float* dwq, float* dwk) {
    __shared__ float s[32][33];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float v = 0.f;
    for (int r = w; r < rows; r += 32) v += __ldcg(part + static_cast<size_t>(r) * 2 * D + col);
    s[w][threadIdx.x & 31] = v;
    __syncthreads();
    if (w != 0) return;
    v = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) v += s[k][threadIdx.x];
    float* dst = col < D ? dwq : dwk;
    if (dst) dst[col % D] = v;
}

}  // namespace elsattn
