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
// around by shuffles.  A tensor with fewer heads than that can put the rows of
// several tokens side by side (MULTI).
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

// Launch shapes, chosen by measurement on 32768 tokens of 32 + 8 heads of 128
// (forward 671 MB, backward 1007 MB moved; a plain copy of that size runs at 6.6 TB/s):
//   forward:  16 warps an SM and 2 steps in flight a warp: 111 us, 6.0 TB/s.  More warps
//             (20: 115 us, 24: 128 us) or more steps in flight (3: 119 us, 5: 128 us) are slower, one
//             step in flight too (138 us).
//   backward: 12 warps an SM, so that a warp's 150-odd registers are held without spills, 2 steps in flight:
//             165 us, 6.1 TB/s (8 warps: 205 us; 16 warps with spills: 216 us).
constexpr int kFwdWarps = 4, kFwdCtasPerSm = 4, kFwdSlots = 3;
constexpr int kBwdWarps = 12, kBwdCtasPerSm = 1, kBwdSlots = 3;

// Quotients of numbers below 2^31 by a divisor that the host knows: with
// 2^(s - 1) < d <= 2^s and m = ceil(2^(31 + s) / d), n / d = (n m) >> (31 + s)
// for every such n (Granlund and Montgomery, division by invariant integers).
// Two instructions; a division takes twenty.
struct Quotient {
    uint32_t m = 0;
    int shift = 0;  // 31 + s - 32
    int d = 1;
    __host__ void set(int divisor) {
        d = divisor;
        int s = 0;
        while ((1ll << s) < divisor) ++s;
        m = s == 0 ? 0u : static_cast<uint32_t>(((1ull << (31 + s)) + divisor - 1) / divisor);
        shift = s - 1;
    }
    __device__ __forceinline__ uint32_t of(uint32_t n) const { return d == 1 ? n : __umulhi(n, m) >> shift; }
};

struct ReadyTensor {
    const __nv_bfloat16* x;   // input rows (backward: the forward's input; unused without a norm)
    const __nv_bfloat16* g;   // backward: gradient of the output rows
    __nv_bfloat16* y;         // output rows (backward: gradient of the input rows)
    const __nv_bfloat16* w;   // [d] norm weight, or nullptr: no norm
    int64_t xs[3], gs[3], ys[3];  // strides in elements: batch, head, token
    int H;
    int hp, tp;               // a warp step holds hp heads (a power of two) of each of tp tokens, hp * tp = rows per warp
    int steps;                // steps of a token (or of tp tokens): ceil(H / hp)
    int steps_per_unit;       // a work unit: so many steps of one token
    Quotient units_per_token; // of a token, or of tp tokens
    uint32_t units;
    float* part;              // backward: [CTAs of this tensor][d] fp32 partial sums of dw, or nullptr
};

struct ReadyParams {
    ReadyTensor t[2];         // Q, K
    int first_k;              // CTAs [0, first_k) work on Q, the others on K
    const int32_t* pos;       // position of token n of batch b on axis a: pos[a * pos_axis + b * pos_batch + n]
    int64_t pos_axis, pos_batch;
    const double* inv_freq;   // [rot / 2]
    int axis_end[kReadyMaxAxes];  // pairs [axis_end[a - 1], axis_end[a]) turn by axis a
    int rot;                  // rotated elements of a row
    Quotient N;
    uint32_t tokens;          // B * N
    bool multi;               // a tensor's steps may hold several tokens (tp > 1)
    float eps;
};

// Packed fp32 pairs: one instruction for two lanes of arithmetic, each
// correctly rounded like the scalar one.
using f2 = uint64_t;
__device__ __forceinline__ f2 pair2(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split2(f2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float sum2(f2 v) {
    float lo, hi;
    split2(v, lo, hi);
    return lo + hi;
}
__device__ __forceinline__ f2 swap2(f2 v) {
    float lo, hi;
    split2(v, lo, hi);
    return pair2(hi, lo);
}

// Eight bf16 as four packed fp32 pairs, and back with one rounding.
__device__ __forceinline__ void unpack8(const uint4& v, f2 (&f)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = pair2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack2(f2 v) {
    float lo, hi;
    split2(v, lo, hi);
    return pack_bf16x2(lo, hi);
}
__device__ __forceinline__ uint4 pack8(const f2 (&f)[4]) { return make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3])); }

// Where lane `c` of a row group has its two vectors, and whether they are rotated.
// Halves: elements 8c.. and rot/2 + 8c.. (the pairs 8c .. 8c + 7); the lanes
// past them hold 16 neighbouring unrotated elements.  Neighbours: elements
// 8c.. and d/2 + 8c.., four pairs each.
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
    // the k-th (0..7) pair of lane c
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
template <int D, bool MULTI>
struct ReadyAngles {
    static constexpr int kLanes = D / 16;        // lanes per row
    static constexpr int kGroups = 32 / kLanes;  // rows per warp step
    static constexpr int kOwn = 8 / kGroups;     // pairs evaluated per lane
    static constexpr int kPos = MULTI ? 8 : kOwn;  // positions held: kOwn for each of a step's tokens
    uint64_t f[kOwn];
    int axis[kOwn];

    // Which pairs, their axes, and their frequencies' loads; finish() converts what arrived.
    template <bool INTER>
    __device__ __forceinline__ void start(const ReadyParams& p, int lane, double (&freq)[kOwn]) {
        const int c = lane % kLanes, g = lane / kLanes;
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            const int i = ReadyLane<D, INTER>::pair(c, g * kOwn + k);
            axis[k] = 0;
            freq[k] = 0.0;
            if (i < (p.rot >> 1)) {
                freq[k] = __ldg(p.inv_freq + i);
#pragma unroll
                for (int a = 0; a < kReadyMaxAxes - 1; ++a) axis[k] += i >= p.axis_end[a] ? 1 : 0;
            }
        }
    }
    __device__ __forceinline__ void finish(const double (&freq)[kOwn]) {
#pragma unroll
        for (int k = 0; k < kOwn; ++k) f[k] = turn_fraction(freq[k]);
    }
    // Positions of the pairs this lane evaluates, for each of the step's tp
    // tokens (issued early).  `at`: where this lane's own token has its positions.
    __device__ __forceinline__ void load(const ReadyParams& p, const ReadyTensor& rt, int64_t at, int (&pos)[kPos]) const {
#pragma unroll
        for (int t = 0; t < (MULTI ? kGroups : 1); ++t) {
            if (MULTI && t >= rt.tp) break;
            const int64_t from = !MULTI || rt.tp == 1 ? at : __shfl_sync(0xffffffffu, at, t * rt.hp * kLanes);
#pragma unroll
            for (int k = 0; k < kOwn; ++k) pos[t * kOwn + k] = p.pos[axis[k] * p.pos_axis + from];
        }
    }
    // cs, sn: of this lane's own token, the step's gt-th
    __device__ __forceinline__ void eval(const int (&pos)[kPos], const ReadyTensor& rt, int gt, int lane, float (&cs)[8],
                                         float (&sn)[8]) const {
#pragma unroll
        for (int t = 0; t < (MULTI ? kGroups : 1); ++t) {
            if (MULTI && t >= rt.tp) break;
            float c0[kOwn], s0[kOwn];
#pragma unroll
            for (int k = 0; k < kOwn; ++k) {
                const uint64_t turn = f[k] * static_cast<uint64_t>(static_cast<int64_t>(pos[t * kOwn + k]));
                // the top 32 bits as a signed fraction of a turn, [-1/2, 1/2); in units of pi: [-1, 1)
                const float x = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f;
                sincospif(x, &s0[k], &c0[k]);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int src = (k / kOwn) * kLanes + lane % kLanes;
                const float cv = __shfl_sync(0xffffffffu, c0[k % kOwn], src);
                const float sv = __shfl_sync(0xffffffffu, s0[k % kOwn], src);
                if (!MULTI || t == 0 || gt == t) {
                    cs[k] = cv;
                    sn[k] = sv;
                }
            }
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

// The turn of a lane's two vectors as coefficients of packed products.  With
// weights w on the inputs (the norm's, or 1) and the angles t:
//   halves:     a' = a (wa cos) + b (-wb sin),  b' = b (wb cos) + a (wa sin)
//   neighbours: v' = v (w cos) + swap(v) (-w_odd sin, w_even sin)   for v = a, b
// so two elements cost two packed operations.  SIGN -1 turns back.
// A vector that is not rotated has cos 1 and sin 0, and its other member is
// replaced by 0: a product of 0 and an infinity must not enter.
template <int D, bool INTER, int SIGN>
struct ReadyTurn {
    f2 ca[4], cb[4], sa[4], sb[4];
    // without weights: the coefficients that are equal share registers
    __device__ __forceinline__ void set(const float (&cs)[8], const float (&sn)[8], bool rot_a, bool rot_b) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (INTER) {  // pair 4 * (vector) + k is the vector's elements 2k, 2k + 1
                const float c0 = rot_a ? cs[k] : 1.f, s0 = rot_a ? SIGN * sn[k] : 0.f;
                const float c1 = rot_b ? cs[4 + k] : 1.f, s1 = rot_b ? SIGN * sn[4 + k] : 0.f;
                ca[k] = pair2(c0, c0);
                cb[k] = pair2(c1, c1);
                sa[k] = pair2(-s0, s0);
                sb[k] = pair2(-s1, s1);
            } else {
                const float s0 = rot_a ? SIGN * sn[2 * k] : 0.f, s1 = rot_a ? SIGN * sn[2 * k + 1] : 0.f;
                ca[k] = cb[k] = pair2(rot_a ? cs[2 * k] : 1.f, rot_a ? cs[2 * k + 1] : 1.f);
                sa[k] = pair2(-s0, -s1);  // of b, in a'
                sb[k] = pair2(s0, s1);    // of a, in b'
            }
        }
    }
    __device__ __forceinline__ void set(const float (&cs)[8], const float (&sn)[8], bool rot_a, bool rot_b,
                                        const f2 (&wa)[4], const f2 (&wb)[4]) {
        set(cs, sn, rot_a, rot_b);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            ca[k] = mul2(wa[k], ca[k]);
            cb[k] = mul2(wb[k], cb[k]);
            sa[k] = mul2(INTER ? swap2(wa[k]) : wb[k], sa[k]);
            sb[k] = mul2(INTER ? swap2(wb[k]) : wa[k], sb[k]);
        }
    }
    // a, b: in place.  all: every lane of the launch rotates (rot == D).
    __device__ __forceinline__ void apply(f2 (&a)[4], f2 (&b)[4], bool all, bool rot_a, bool rot_b) const {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f2 oa = INTER ? swap2(a[k]) : b[k], ob = INTER ? swap2(b[k]) : a[k];
            if (!all) {
                oa = rot_a ? oa : 0;
                ob = rot_b ? ob : 0;
            }
            a[k] = fma2(oa, sa[k], mul2(a[k], ca[k]));
            b[k] = fma2(ob, sb[k], mul2(b[k], cb[k]));
        }
    }
};

// This CTA's tensor and its place among that tensor's CTAs.
struct ReadyPlace {
    int t, block, blocks;
    __device__ __forceinline__ explicit ReadyPlace(const ReadyParams& p) {
        t = static_cast<int>(blockIdx.x) >= p.first_k ? 1 : 0;
        block = t ? blockIdx.x - p.first_k : blockIdx.x;
        blocks = t ? gridDim.x - p.first_k : p.first_k;
    }
};

__device__ __forceinline__ void load_weight(const __nv_bfloat16* w, int a0, int b0, f2 (&wa)[4], f2 (&wb)[4]) {
    if (w) {
        unpack8(*reinterpret_cast<const uint4*>(w + a0), wa);
        unpack8(*reinterpret_cast<const uint4*>(w + b0), wb);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) wa[k] = wb[k] = pair2(1.f, 1.f);
    }
}

// A warp's walk over its units, step by step, seen by one lane: where the
// step has its row.
template <int GROUPS, bool MULTI>
struct ReadyWalk {
    uint32_t u;   // unit (>= units: done)
    int s, s1;    // step within the token, and the unit's end
    int gh, gt;   // this lane's head and token within a step
    int b, n;     // its token's batch and place
    bool live;    // the token exists
    __device__ __forceinline__ void begin(const ReadyTensor& rt, uint32_t unit, int g) {
        u = unit;
        gh = MULTI ? g & (rt.hp - 1) : g;
        gt = MULTI ? g / rt.hp : 0;
    }
    __device__ __forceinline__ void decode(const ReadyParams& p, const ReadyTensor& rt) {
        const uint32_t group = rt.units_per_token.of(u);
        s = static_cast<int>(u - group * rt.units_per_token.d) * rt.steps_per_unit;
        s1 = min(rt.steps, s + rt.steps_per_unit);
        uint32_t token = MULTI ? group * rt.tp + gt : group;
        live = !MULTI || token < p.tokens;
        if (!live) token = p.tokens - 1;
        b = static_cast<int>(p.N.of(token));
        n = static_cast<int>(token - static_cast<uint32_t>(b) * p.N.d);
    }
    __device__ __forceinline__ bool on(const ReadyTensor& rt, int step) const { return live && step * GROUPS + gh < rt.H; }
    __device__ __forceinline__ int64_t offset(const int64_t (&st)[3]) const {
        return b * st[0] + (s * GROUPS + gh) * st[1] + n * st[2];
    }
    __device__ __forceinline__ int64_t positions(const ReadyParams& p) const { return b * p.pos_batch + n; }
};

// 16 bytes from global to shared memory, asynchronously; zeros where !on.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

// One warp's rows in flight: a ring of U steps in shared memory, filled by
// asynchronous copies that run ahead over the ends of units.  Each lane reads
// back only what it copied itself, so its own wait is all the synchronisation.
// U slots, U - 1 steps in flight: a step's copies go to the slot read one step
// before, whose values have been used (its results are stored) by then.
// VECS: 16-byte vectors a lane moves per step.
template <int D, int VECS, int U, bool MULTI>
struct ReadyRing {
    using A = ReadyAngles<D, MULTI>;
    static constexpr int kBytes = U * VECS * 512;  // per warp
    ReadyWalk<A::kGroups, MULTI> w;
    uint32_t base;       // this lane's place in the warp's ring
    uint32_t warps;
    int fill, slot;      // the ring slots to fill and to read next
    const __nv_bfloat16 *x, *g;   // the next step's rows (g: the second source, where there is one)

    __device__ __forceinline__ void place(const ReadyTensor& rt, bool first, bool second) {
        if (first) x = rt.x + w.offset(rt.xs);
        if (second) g = rt.g + w.offset(rt.gs);
    }
    template <class Lane>
    __device__ __forceinline__ void issue(const ReadyParams& p, const ReadyTensor& rt, const Lane& at, bool first,
                                          bool second) {
        if (w.u < rt.units) {
            const bool on = w.on(rt, w.s);
            const uint32_t dst = base + fill * (VECS * 512);
            if (first) {
                copy16(dst, on ? x + at.a0 : rt.x, on);
                copy16(dst + 512, on ? x + at.b0 : rt.x, on);
                x += A::kGroups * rt.xs[1];
            }
            if (second) {
                copy16(dst + (VECS - 2) * 512, on ? g + at.a0 : rt.g, on);
                copy16(dst + (VECS - 1) * 512, on ? g + at.b0 : rt.g, on);
                g += A::kGroups * rt.gs[1];
            }
            if (++w.s == w.s1) {
                w.u += warps;
                if (w.u < rt.units) {
                    w.decode(p, rt);
                    place(rt, first, second);
                }
            }
        }
        copy_commit();
        fill = fill + 1 == U ? 0 : fill + 1;
    }
    // Waits for the next step's rows; returns where they are.
    __device__ __forceinline__ uint32_t next() {
        copy_wait<U - 2>();
        const uint32_t a = base + slot * (VECS * 512);
        slot = slot + 1 == U ? 0 : slot + 1;
        return a;
    }
    template <class Lane>
    __device__ __forceinline__ void start(const ReadyParams& p, const ReadyTensor& rt, const Lane& at, int grp, bool first,
                                          bool second, uint32_t smem, uint32_t u0, uint32_t n) {
        base = smem + (threadIdx.x & 31) * 16;
        warps = n;
        fill = slot = 0;
        x = g = nullptr;
        w.begin(rt, u0, grp);
        if (w.u < rt.units) {
            w.decode(p, rt);
            place(rt, first, second);
        }
#pragma unroll 1
        for (int i = 0; i < U - 1; ++i) issue(p, rt, at, first, second);
    }
};

extern __shared__ __align__(16) uint8_t ready_smem[];

// U: slots of a warp's ring.
template <int D, bool INTER, int U, bool MULTI>
__global__ void __launch_bounds__(kFwdWarps * 32, kFwdCtasPerSm) qk_norm_rope_kernel(const __grid_constant__ ReadyParams p) {
    using A = ReadyAngles<D, MULTI>;
    using Ring = ReadyRing<D, 2, U, MULTI>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = lane % A::kLanes, g = lane / A::kLanes;
    const ReadyLane<D, INTER> at(c, p.rot);
    const ReadyPlace place(p);
    const ReadyTensor& rt = p.t[place.t];
    const uint32_t warps = place.blocks * kFwdWarps;
    ReadyWalk<A::kGroups, MULTI> w;
    w.begin(rt, place.block * kFwdWarps + warp, g);
    if (w.u >= rt.units) return;
    // every load that the first rows wait for is under way before any of it is used
    A angles;
    double freq[A::kOwn];
    angles.template start<INTER>(p, lane, freq);
    w.decode(p, rt);
    int pos[A::kPos];
    angles.load(p, rt, w.positions(p), pos);
    Ring ring;
    ring.start(p, rt, at, g, true, false, smem_u32(ready_smem) + warp * Ring::kBytes, w.u, warps);
    angles.finish(freq);
    const bool norm = rt.w != nullptr, all = p.rot == D;
    while (true) {
        float cs[8], sn[8];
        angles.eval(pos, rt, w.gt, lane, cs, sn);
        ReadyTurn<D, INTER, 1> turn;
        {  // the weights are read again for each unit (from L1): 16 registers less
            f2 wa[4], wb[4];
            load_weight(rt.w, at.a0, at.b0, wa, wb);
            turn.set(cs, sn, at.rot_a, at.rot_b, wa, wb);
        }
        __nv_bfloat16* dst = rt.y + w.offset(rt.ys);
        int s = w.s;
        const int s1 = w.s1;
        const bool live = w.live;
        w.u += warps;
        const bool more = w.u < rt.units;
        if (more) {  // the next unit's positions arrive while this one's rows are worked on
            w.decode(p, rt);
            angles.load(p, rt, w.positions(p), pos);
        }
        for (; s < s1; ++s) {
            f2 a[4], bb[4];
            const uint32_t src = ring.next();
            unpack8(ld_shared16(src), a);
            unpack8(ld_shared16(src + 512), bb);
            ring.issue(p, rt, at, true, false);
            if (norm) {
                f2 s2 = mul2(a[0], a[0]), t2 = mul2(bb[0], bb[0]);
#pragma unroll
                for (int k = 1; k < 4; ++k) {
                    s2 = fma2(a[k], a[k], s2);
                    t2 = fma2(bb[k], bb[k], t2);
                }
                const float r = rsqrtf(row_sum<A::kLanes>(sum2(s2) + sum2(t2)) * (1.0f / D) + p.eps);
                const f2 r2 = pair2(r, r);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    a[k] = mul2(a[k], r2);
                    bb[k] = mul2(bb[k], r2);
                }
            }
            turn.apply(a, bb, all, at.rot_a, at.rot_b);
            if (live && s * A::kGroups + w.gh < rt.H) {
                *reinterpret_cast<uint4*>(dst + at.a0) = pack8(a);
                *reinterpret_cast<uint4*>(dst + at.b0) = pack8(bb);
            }
            dst += A::kGroups * rt.ys[1];
        }
        if (!more) break;
    }
}

// The gradient.  dw is summed per lane in fp32 over the warp's rows, then over
// the row groups of the warp, the warps of the CTA (both in a fixed order), and
// by qk_norm_rope_dw_kernel over the CTAs: the same inputs give the same bits.
template <int D, bool INTER, int U, bool MULTI>
__global__ void __launch_bounds__(kBwdWarps * 32, kBwdCtasPerSm) qk_norm_rope_bwd_kernel(const __grid_constant__ ReadyParams p) {
    using A = ReadyAngles<D, MULTI>;
    using Ring = ReadyRing<D, 4, U, MULTI>;
    __shared__ float s_dw[kBwdWarps][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = lane % A::kLanes, g = lane / A::kLanes;
    const ReadyLane<D, INTER> at(c, p.rot);
    const ReadyPlace place(p);
    const ReadyTensor& rt = p.t[place.t];
    const bool norm = rt.w != nullptr, all = p.rot == D;
    const uint32_t warps = place.blocks * kBwdWarps;
    f2 acc[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = 0;
    ReadyWalk<A::kGroups, MULTI> w;
    w.begin(rt, place.block * kBwdWarps + warp, g);
    bool more = w.u < rt.units;
    if (more) {
        A angles;
        double freq[A::kOwn];
        angles.template start<INTER>(p, lane, freq);
        w.decode(p, rt);
        int pos[A::kPos];
        angles.load(p, rt, w.positions(p), pos);
        f2 wa[4], wb[4];
        load_weight(rt.w, at.a0, at.b0, wa, wb);
        Ring ring;
        ring.start(p, rt, at, g, norm, true, smem_u32(ready_smem) + warp * Ring::kBytes, w.u, warps);
        angles.finish(freq);
        while (more) {
            float cs[8], sn[8];
            angles.eval(pos, rt, w.gt, lane, cs, sn);
            ReadyTurn<D, INTER, -1> turn;
            turn.set(cs, sn, at.rot_a, at.rot_b);
            __nv_bfloat16* dst = rt.y + w.offset(rt.ys);
            int s = w.s;
            const int s1 = w.s1;
            const bool live = w.live;
            w.u += warps;
            more = w.u < rt.units;
            if (more) {
                w.decode(p, rt);
                angles.load(p, rt, w.positions(p), pos);
            }
            for (; s < s1; ++s) {
                const bool on = live && s * A::kGroups + w.gh < rt.H;
                f2 ua[4], ub[4], ha[4], hb[4];
                const uint32_t src = ring.next();
                unpack8(ld_shared16(src + 1024), ua);
                unpack8(ld_shared16(src + 1536), ub);
                if (norm) {
                    unpack8(ld_shared16(src), ha);
                    unpack8(ld_shared16(src + 512), hb);
                }
                ring.issue(p, rt, at, norm, true);
                turn.apply(ua, ub, all, at.rot_a, at.rot_b);
                if (norm) {
                    f2 va[4], vb[4];
                    f2 s2 = 0, d2 = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        s2 = fma2(ha[k], ha[k], fma2(hb[k], hb[k], s2));
                        va[k] = mul2(ua[k], wa[k]);
                        vb[k] = mul2(ub[k], wb[k]);
                        d2 = fma2(va[k], ha[k], fma2(vb[k], hb[k], d2));
                    }
                    // a lane without a row adds nothing to dw, also where eps is 0
                    const float rr = rsqrtf(row_sum<A::kLanes>(sum2(s2)) * (1.0f / D) + p.eps);
                    const float r = on ? rr : 0.f;
                    const float m = row_sum<A::kLanes>(sum2(d2)) * r * (1.0f / D);  // mean(u w h)
                    const f2 r2 = pair2(r, r), m2 = pair2(-m, -m);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        ha[k] = mul2(ha[k], r2);
                        hb[k] = mul2(hb[k], r2);
                        acc[k] = fma2(ua[k], ha[k], acc[k]);
                        acc[4 + k] = fma2(ub[k], hb[k], acc[4 + k]);
                        ua[k] = mul2(r2, fma2(ha[k], m2, va[k]));
                        ub[k] = mul2(r2, fma2(hb[k], m2, vb[k]));
                    }
                }
                if (on) {
                    *reinterpret_cast<uint4*>(dst + at.a0) = pack8(ua);
                    *reinterpret_cast<uint4*>(dst + at.b0) = pack8(ub);
                }
                dst += A::kGroups * rt.ys[1];
            }
        }
    }
    if (!rt.part) return;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float v[2];
        split2(acc[k], v[0], v[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int off = 16; off >= A::kLanes; off >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
            if (g == 0) s_dw[warp][(k < 4 ? at.a0 + 2 * k : at.b0 + 2 * (k - 4)) + i] = v[i];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += blockDim.x) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kBwdWarps; ++k) v += s_dw[k][i];
        rt.part[static_cast<size_t>(place.block) * D + i] = v;
    }
}

// dw of both tensors from their CTAs' partial sums: CTA (x, y) has 32 columns
// of tensor y, whose rows are dealt to 32 warps and added in a fixed order.
struct ReadyDw {
    const float* part[2];
    int rows[2];
    float* dw[2];
};
template <int D>
__global__ void __launch_bounds__(1024) qk_norm_rope_dw_kernel(const ReadyDw a) {
    __shared__ float s[32][33];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5, t = blockIdx.y;
    if (!a.dw[t]) return;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float v = 0.f;
    for (int r = w; r < a.rows[t]; r += 32) v += __ldcg(a.part[t] + static_cast<size_t>(r) * D + col);
    s[w][threadIdx.x & 31] = v;
    __syncthreads();
    if (w != 0) return;
    v = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) v += s[k][threadIdx.x];
    a.dw[t][col] = v;
}

}  // namespace elsattn
