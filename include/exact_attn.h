/*
 * exact_attn.h - C ABI of the GB300 (sm_103a) exact self-attention forward.
 *
 * The operation is the attention graph of "From Attention Graph to
 * FlashAttention - A Memory-Centric Compilation Approach in AICF", section 1
 * (Introduction): the query-key products, masked, normalised row by row with
 * a softmax and applied to the values,
 *     O = softmax(mask(scale * Q K^T)) V,
 * plus the per-row log-sum-exp
 *     LSE_i = ln sum_j exp(scale * q_i . k_j)   (over the keys the mask keeps).
 * It is computed as the streaming pass of section 3 of that page: a query
 * tile stays on chip while the K/V tiles stream past it, each contributing its
 * scores to a running softmax and to the output, so the N x N score and
 * probability matrices never reach device memory.  The library is the
 * `flash_attention(Q, K, V)` call of section 4 of the same page, with the
 * optional mask of section 5 as a flag.
 *
 * Conventions for every entry point:
 *   - Q, K, V, O are bf16 tensors laid out [B, H, N, d], contiguous, d fastest;
 *     LSE is fp32 [B, H, N].  All five live in device memory, are owned by the
 *     caller and must not overlap (not checked).
 *   - causal != 0 keeps key j for query i iff j <= i; masked scores are
 *     -infinity, i.e. they drop out of the softmax.
 *   - Calls are asynchronous on `stream` and never synchronise it.
 *   - Errors are returned as attn_status codes; nothing aborts or throws
 *     across this boundary.
 */
#ifndef EXACT_ATTN_H
#define EXACT_ATTN_H

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ATTN_OK = 0,
    ATTN_ERR_INVALID_ARG = 1,  /* null pointer, bad size, or a scale out of range (see each call) */
    ATTN_ERR_UNSUPPORTED = 2,  /* head dim other than 64/128, or a device other than sm_103 */
    ATTN_ERR_MISALIGNED = 3,   /* a tensor base address is not 16-byte aligned */
    ATTN_ERR_CUDA = 4,         /* a CUDA runtime/driver call failed: see attn_last_cuda_error() */
    ATTN_ERR_TIMEOUT = 5,      /* a kernel-side wait ran out of time (reported by attn_last_device_error) */
    ATTN_ERR_NO_DEVICE = 6     /* no CUDA device is visible */
} attn_status;

/*
 * Tile plan chosen by the I/O-count planner (see attn_plan).  Sizes are in
 * elements unless named *_bytes.
 */
typedef struct {
    int Br;               /* query rows per tile (the tcgen05 M dimension) */
    int Bc;               /* keys per streamed K/V tile */
    int q_tiles;          /* query tiles resident per CTA (they share every K/V tile) */
    int kv_stages;        /* depth of the shared-memory K/V ring (one tile per stage) */
    int tmem_cols;        /* tensor-memory columns allocated per CTA */
    int smem_bytes;       /* dynamic shared memory per CTA */
    int threads;          /* threads per CTA */
    int num_units;        /* work units: (batch*head, group of q_tiles query tiles) */
    int grid;             /* persistent CTAs launched (<= SM count) */
    int heads_per_group;  /* causal schedule: heads interleaved per scheduling group */
    double flops;         /* 4*B*H*N^2*d, halved when causal */
    double io_bytes;      /* Theta(N*d) bound: bf16 Q,K,V read + bf16 O, fp32 LSE written once */
    double l2_bytes;      /* modelled L2->SMEM traffic of the chosen tiling */
    double hbm_bytes;     /* modelled HBM traffic: io_bytes, plus the K/V re-reads that miss L2 when
                             the K/V of the heads in flight exceed the L2 budget */
    int io_opt_q_tiles;   /* the tiling with least L2->SMEM traffic among those the SM runs at the   */
    int io_opt_Bc;        /* full tensor rate within its shared memory, tensor memory and registers */
    double io_opt_l2_bytes; /* its modelled L2->SMEM traffic (the kernel runs this tiling) */
    double kv_in_flight_bytes; /* K/V bytes of the heads the schedule streams at the same time */
    double l2_fit;        /* fraction of those that fit the L2 budget (1: every head's K/V read once) */
} attn_plan_t;

/*
 * attn_fwd - O = softmax(scale * Q K^T + mask) V and LSE, for B*H independent
 * (batch, head) problems.
 *   Q, K, V : const bf16 [B,H,N,d] device pointers, 16-byte aligned
 *   O       : bf16 [B,H,N,d] device pointer, 16-byte aligned (written)
 *   LSE     : fp32 [B,H,N] device pointer, 4-byte aligned (written; natural log)
 *   B, H, N : >= 1 with B*H*N < 2^31;  d : 64 or 128
 *   causal  : 0 = no mask, nonzero = causal mask (key j visible to query i iff j <= i)
 *   scale   : any finite value (typically 1/sqrt(d)).  A negative scale is run
 *             as |scale| on the negated scores (the tensor core's negate bit), so
 *             the running maximum tracks the largest scaled score; zero gives
 *             the plain average of the visible values (LSE = ln #visible).
 *   stream  : CUDA stream on the current device (0 = legacy default stream)
 * Returns ATTN_OK when the launch was queued.  Kernel-side timeouts are
 * reported later by attn_last_device_error().
 */
int attn_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H, int N, int d,
             int causal, float scale, cudaStream_t stream);

/*
 * attn_fwd_host - the same operation on HOST buffers: copies Q, K, V to the
 * device, runs attn_fwd and copies O and LSE back.  The work is split into up
 * to 8 chunks of (batch, head) pairs whose copies in, kernels and copies out
 * run on the library's own per-device streams, so transfers overlap compute:
 * each chunk's kernel starts once its inputs are in, and the copies out start
 * once every copy in has landed (the two directions share the host link).
 * It is ordered after the work already queued on `stream`, and `stream` waits
 * for the last copy out.  Pinned host memory makes the copies asynchronous.
 * The caller synchronises `stream` before reading O / LSE.  Calls from several
 * host threads are serialised while they queue their work.
 *   Qh, Kh, Vh, Oh, LSEh : host pointers with the layouts of attn_fwd
 *   workspace            : device buffer of at least attn_fwd_host_workspace_bytes()
 *                          bytes, 16-byte aligned, owned by the caller
 */
int attn_fwd_host(const void* Qh, const void* Kh, const void* Vh, void* Oh, float* LSEh, int B, int H, int N,
                  int d, int causal, float scale, void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Device bytes attn_fwd_host needs for its staging copies of Q, K, V, O, LSE. */
size_t attn_fwd_host_workspace_bytes(int B, int H, int N, int d);

/*
 * attn_fwd_split - attn_fwd with a work schedule chosen for the launch's shape.
 * A work unit is a pair of 128-row query tiles of one (batch, head) against
 * every key they see.
 *   - Fewer units than SMs (few heads, or a causal mask whose longest query
 *     tiles dominate): the K/V range of the heaviest units is cut into
 *     segments, either run on the SMs the units leave idle (one wave), or,
 *     for a causal mask, claimed dynamically with the other units (below),
 *     whichever the host's schedule estimate finds shorter.
 *   - More equal units than SMs (no mask): the units of the last, partial wave
 *     are cut into segments that spread over all SMs.
 *   - More causal units than SMs (units of unequal length): no segments; the
 *     persistent CTAs claim units dynamically, heaviest first, from a counter
 *     in `workspace`.  Every unit is computed exactly as by attn_fwd, so the
 *     outputs are bit-identical to it.
 * A segment is a work item of its own: it writes its partial result (O over
 * the segment's keys, normalised, fp32, and that segment's LSE) to `workspace`
 * (with an L2 evict-last policy), and a second kernel on `stream` merges the
 * segments of each row by
 *     LSE = log sum_s exp(LSE_s),  O = sum_s exp(LSE_s - LSE) O_s,
 * the combination step of the online softmax (the streaming reformulation of
 * the IO-Aware Algorithms page) applied across segments, then drops the
 * partial rows from L2 without writing them back.  The result is the same
 * operation as attn_fwd, up to floating-point rounding.  Launches on `stream`:
 * a one-thread kernel that zeroes the schedule counter (dynamic schedule only;
 * the attention kernel is its programmatic dependent and waits for it only
 * before its first claim), the attention kernel, and the combine kernel (split
 * launches only).
 *   arguments as attn_fwd, plus
 *   workspace       : device buffer of at least attn_fwd_split_workspace_bytes()
 *                     bytes, 16-byte aligned, owned by the caller, not used by
 *                     other work while this call runs; may be NULL when that
 *                     size is 0 (this call then runs exactly attn_fwd)
 *   workspace_bytes : its size
 * Returns ATTN_ERR_INVALID_ARG when a workspace is needed and it is missing,
 * misaligned or too small; otherwise as attn_fwd.
 */
int attn_fwd_split(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H, int N, int d,
                   int causal, float scale, void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Workspace bytes attn_fwd_split needs on the current device; 0 when it needs
 * none (or the shape is invalid). */
size_t attn_fwd_split_workspace_bytes(int B, int H, int N, int d, int causal);

/* K/V segments per split unit that attn_fwd_split chooses on the current
 * device: 1 when it does not split, 0 for an invalid shape or no device. */
int attn_fwd_split_segments(int B, int H, int N, int d, int causal);

/*
 * attn_fwd_split_choice - host only: the work split attn_fwd_split would use on
 * a device with num_sms SMs.  Writes the segments per split unit (1: no split),
 * the first split unit and the number of split units (in the kernel's unit
 * order), and whether the dynamic schedule is used (0 or 1).  Returns
 * ATTN_ERR_INVALID_ARG for a null pointer, num_sms < 1 or a shape out of range,
 * ATTN_ERR_UNSUPPORTED for d other than 64 or 128.
 */
int attn_fwd_split_choice(int B, int H, int N, int d, int causal, int num_sms, int* segs, int* first, int* units,
                          int* dynamic);

/*
 * attn_bwd - gradients of attn_fwd for an upstream gradient dO of O:
 *     dV = P^T dO,  dS = P * (dO V^T - D) with D_i = sum_c dO_ic O_ic,
 *     dQ = scale * dS K,  dK = scale * dS^T Q,
 * where P = softmax(scale * Q K^T + mask) is recomputed from Q, K and the
 * forward's LSE instead of being stored (FlashAttention's recomputation in the
 * backward pass, "IO-Aware Algorithms").  No gradient flows into LSE.
 *   Q, K, V, O, dO : const bf16 [B,H,N,d] device pointers (O and LSE as written
 *                    by attn_fwd for the same Q, K, V, causal, scale)
 *   LSE            : const fp32 [B,H,N]
 *   dQ, dK, dV     : bf16 [B,H,N,d] device pointers (written)
 *   workspace      : device buffer of at least attn_bwd_workspace_bytes() bytes,
 *                    16-byte aligned, owned by the caller: the fp32 dQ accumulator
 *                    [B,H,N,d], then the row statistics -scale * D and
 *                    -LSE * log2(e) (negated for the kernel's packed FMAs) on rows
 *                    padded to a multiple of 128 per (batch, head)
 * Same size, alignment, scale and error rules as attn_fwd; asynchronous on `stream`.
 */
int attn_bwd(const void* Q, const void* K, const void* V, const void* O, const float* LSE, const void* dO, void* dQ,
             void* dK, void* dV, int B, int H, int N, int d, int causal, float scale, void* workspace,
             size_t workspace_bytes, cudaStream_t stream);

/* Device bytes attn_bwd needs as workspace:
 * align256(4*B*H*N*d) + 2 * align256(4*B*H*ceil(N/128)*128); 0 for a
 * non-positive size. */
size_t attn_bwd_workspace_bytes(int B, int H, int N, int d);

/*
 * attn_plan - host only, launches nothing.  Fills *out with the tiling the
 * planner derives from an I/O count of the two tall-and-skinny products
 * (S = Q K^T and O = P V): the least-traffic tiling among those an sm_103 SM
 * holds (shared memory, tensor memory, registers) and runs at the full tensor
 * rate (the I/O-optimal tiling of the AttenIO abstract, "I/O Analysis is All
 * You Need", ASPLOS 2026).  That is the tiling the kernel is compiled for;
 * ATTN_ERR_UNSUPPORTED if it ever were not.  num_sms <= 0 queries the current
 * device.
 */
int attn_plan(int B, int H, int N, int d, int causal, int num_sms, attn_plan_t* out);

/*
 * attn_last_device_error - synchronises `stream`, then reads and clears the
 * current device's kernel error word.  Returns ATTN_OK or ATTN_ERR_TIMEOUT.
 */
int attn_last_device_error(cudaStream_t stream);

/* The cudaError_t of the most recent ATTN_ERR_CUDA on this thread (0 if none). */
int attn_last_cuda_error(void);

/* A static, human-readable description of a status code. */
const char* attn_strerror(int status);

/*
 * attn_debug_wait_timeout - test hook for the bounded-wait machinery: launches
 * one CTA that waits on an mbarrier nobody arrives on, with the given limit in
 * nanoseconds (<= 10 s).  The kernel gives up, records ATTN_ERR_TIMEOUT in the
 * device error word and exits normally, so the context stays usable; read the
 * result with attn_last_device_error().
 */
int attn_debug_wait_timeout(uint64_t timeout_ns, cudaStream_t stream);

/*
 * attn_debug_arm_timeout - test hook for the kernels' own abort path
 * (every wait is bounded: a role whose wait runs out records ATTN_ERR_TIMEOUT,
 * the other roles leave their loops, in-flight copies and MMAs are drained
 * and tensor memory is freed before the kernel returns).  Arms a one-shot:
 * the next forward launch of this process (attn_fwd, attn_fwd_split,
 * attn_fwd_noalloc; the first chunk of attn_fwd_host; attn_fwd_packed,
 * attn_bwd_packed, attn_fwd_tree) runs with a wait limit
 * of timeout_ns (1 us .. 1 s) instead of 4 s, and its CTA 0 (of the packed and
 * paged calls each even CTA that has work) arms the barrier
 * of its first query-tile copy without issuing the copy, so the wait on it
 * runs out.  That launch's outputs are left partly unwritten; the status is
 * read with attn_last_device_error() (attn_noalloc_last_device_error() after
 * attn_fwd_noalloc).  Launches after it are normal.  ATTN_ERR_INVALID_ARG for
 * a limit out of range.  Not for production use.
 */
int attn_debug_arm_timeout(uint64_t timeout_ns);

/*
 * attn_fwd_noalloc - attn_fwd for callers that must not let the library
 * allocate device memory: applications that reserve all of device memory for
 * their own pool up front (such as a server handing the rest of HBM to its
 * cache), or that cannot afford the implicit device synchronisation of
 * cudaMalloc on their path.  The paper has no counterpart; it is an interface
 * variant of attn_fwd with the same arguments, layouts and results.
 *
 * The kernel's only scratch memory is its 4-byte error word.  attn_fwd keeps
 * it in a block the library allocates on first use; this entry point keeps it
 * instead in a fixed 256-byte array compiled into the library (a static
 * __device__ array), which every device that loads the library holds until
 * exit.  The scratch a call needs does not grow with B, H, N or d; a
 * requirement above 256 bytes would be rejected with ATTN_ERR_INVALID_ARG.
 *   - It calls no cudaMalloc, cudaFree or other allocating routine.
 *   - The first call on a device also does that device's one-time set-up
 *     (it looks up the array's device address and sets the kernel's
 *     shared-memory limit); make that first call before any stream capture.
 *   - Every call shares the one array and clears its error word before the
 *     launch.  Calls that overlap on the GPU (other streams, other threads)
 *     race on that word; serialise them.
 *   - A kernel-side timeout is recorded in the array: read it with
 *     attn_noalloc_last_device_error() before the next call clears it.
 * Returns the same status codes as attn_fwd.
 */
int attn_fwd_noalloc(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H, int N, int d,
                     int causal, float scale, cudaStream_t stream);

/*
 * attn_noalloc_last_device_error - the error word of attn_fwd_noalloc: waits
 * for `stream`, then reads the word in the fixed array and clears it (an
 * asynchronous copy and memset on `stream`, each waited for); allocates
 * nothing.  Returns ATTN_OK or ATTN_ERR_TIMEOUT for the most recent
 * attn_fwd_noalloc on the current device, or a set-up error (as attn_fwd_noalloc).
 */
int attn_noalloc_last_device_error(cudaStream_t stream);

/*
 * attn_fwd_fp8 - the same forward on 8-bit inputs (the FP8 variant that the
 * quantisation effects of the Neural Circuit Graph (NCG) abstract's
 * performance modelling motivate: halved I/O and twice the tensor-core rate).  Q, K and V are given as
 * E4M3 codes (OCP 8-bit floating point, E4M3: 1 sign, 4 exponent bits with
 * bias 7, 3 mantissa bits) with one fp32 scale per tensor; the real inputs are
 * q_scale * e4m3(Q8) and likewise K, V.  Computes
 *     O = softmax(scale * Q K^T + mask) V   (bf16 [B,H,N,d]),  LSE (fp32 [B,H,N])
 * with S accumulated in fp32 from the exact code products, P rounded to E4M3
 * and staged in shared memory for the second product, and O / l in fp32.
 * Causal launches with more work units than SMs run a dynamic schedule: CTAs
 * claim units, heaviest first, from a counter in `workspace` that this call
 * zeroes on `stream`; each unit is computed as under the static schedule.
 *   Q8, K8, V8 : const uint8 [B,H,N,d] E4M3 codes, device, 16-byte aligned
 *   O, LSE     : as attn_fwd
 *   scale, q_scale, k_scale, v_scale : finite and > 0
 *   workspace  : device buffer of at least attn_fwd_fp8_workspace_bytes(), 16-byte
 *                aligned, owned by the caller, not used by other work while this
 *                call runs: V transposed to [B,H,d,N] (rows padded to 16 bytes),
 *                then the schedule counter, written by this call
 * d must be 128 (ATTN_ERR_UNSUPPORTED otherwise).  Launches on `stream`: the
 * transpose of V, then the attention kernel; under the dynamic schedule a
 * one-thread kernel zeroing the schedule counter comes between them, and a
 * split launch ends with the combine kernel.  The same argument, size and error
 * rules as attn_fwd otherwise.
 */
int attn_fwd_fp8(const void* Q8, const void* K8, const void* V8, void* O, float* LSE, int B, int H, int N, int d,
                 int causal, float scale, float q_scale, float k_scale, float v_scale, void* workspace,
                 size_t workspace_bytes, cudaStream_t stream);

/* Device bytes attn_fwd_fp8 needs as workspace: B*H*d*ceil16(N) rounded up to 256,
 * plus 256 for the schedule counter; 0 for a non-positive size. */
size_t attn_fwd_fp8_workspace_bytes(int B, int H, int N, int d);

/*
 * attn_softmax_rows - standalone streaming row softmax ("Softmax streaming",
 * section 8 of "From Attention Graph to FlashAttention - A Memory-Centric
 * Compilation Approach in AICF"):
 *     Y[r, i] = exp(X[r, i] - max_j X[r, j]) / sum_j exp(X[r, j] - max_j X[r, j])
 * with the row statistics gathered in one pass by the online-softmax
 * recurrence and fp32 arithmetic.
 *   X, Y      : bf16 [R, N] row-major device arrays, 16-byte aligned (may alias: in place is allowed)
 *   R, N      : 1 <= R < 2^31; N >= 1 and a multiple of 8 (ATTN_ERR_UNSUPPORTED otherwise)
 *   workspace : needed when N > 65536: attn_softmax_rows_workspace_bytes() bytes,
 *               8-byte aligned, owned by the caller; may be NULL otherwise
 * Rows of N <= 65536 are held by one CTA; rows of up to 4 * 65536 by a
 * thread-block cluster of ceil(N / 65536) CTAs that exchange their partial
 * statistics through distributed shared memory: both read X once and write Y
 * once.  Longer rows (or a device that cannot hold the cluster) are handled in
 * segments of 16384 with a second read of X, using the workspace for the
 * per-segment statistics.  Asynchronous on `stream`.
 */
int attn_softmax_rows(const void* X, void* Y, int64_t R, int N, void* workspace, size_t workspace_bytes,
                      cudaStream_t stream);

/* Device bytes attn_softmax_rows needs as workspace (0 when N <= 65536). */
size_t attn_softmax_rows_workspace_bytes(int64_t R, int N);

/*
 * attn_layernorm_rows - standalone streaming layer normalisation ("LayerNorm
 * streaming", same section): per row,
 *     mean = sum_j x_j / N,  var = sum_j (x_j - mean)^2 / N,
 *     Y[r, i] = (X[r, i] - mean) / sqrt(var + eps) * gamma[i] + beta[i],
 * the statistics gathered in one pass (running mean and sum of squared
 * deviations, merged pairwise) in fp32.
 *   X, Y        : bf16 [R, N] row-major device arrays, 16-byte aligned (in place is allowed)
 *   gamma, beta : bf16 [N] device arrays, 16-byte aligned
 *   R, N        : 1 <= R < 2^31; N a multiple of 8, at most 65536 (ATTN_ERR_UNSUPPORTED otherwise)
 *   eps         : finite, >= 0
 * Each row is read once and written once.  Asynchronous on `stream`.
 */
int attn_layernorm_rows(const void* X, const void* gamma, const void* beta, void* Y, int64_t R, int N, float eps,
                        cudaStream_t stream);

/*
 * attn_qk_norm_rope - queries and keys made ready for attn_fwd: per token and
 * head, the RMS norm of the row and the rotation by the token's position, in
 * one pass over Q and K (the fusion the "IO-Aware Algorithms" page asks of
 * memory-bound steps: one read and one write).  In fp32,
 *     y = x / sqrt(mean_j x_j^2 + eps) * weight        (a null weight: y = x),
 *     (y_a, y_b) -> (y_a cos t - y_b sin t, y_b cos t + y_a sin t)
 * for each rotated pair, t = position[axis(i)] * inv_freq[i] for pair i;
 * elements past the rotated ones keep y.  Rounded to bf16 once, at the end.
 * The angle is exact modulo a turn for every int32 position, up to the
 * rounding of inv_freq / (2 pi) to 2^-53 of a turn (times the position).
 * The sum of squares is fp32 too: it overflows for rows with elements beyond about
 * 1e18, which give 0, and with eps = 0 it loses its digits for rows below about 1e-19.
 *   Q, Qout : bf16 [B, Hq, N, d] device views, d fastest, 16-byte aligned
 *   K, Kout : bf16 [B, Hk, N, d] device views; Hq and Hk are independent
 *   *_strides : host arrays of three strides in elements (batch, head, token),
 *             multiples of 8 (ATTN_ERR_MISALIGNED), copied by the call; NULL for
 *             a contiguous tensor.  So Q and K may be slices of a projection's
 *             output [B, N, ...] and the outputs rows of a cache.  An input stride may
 *             be 0 (a broadcast axis); a written axis longer than 1 may not
 *             (ATTN_ERR_INVALID_ARG).  In place (an output with its input's
 *             address and strides) is allowed, any other overlap is not (not checked).
 *   q_weight, k_weight : bf16 [d] device, 16-byte aligned, or NULL: that tensor is only rotated
 *   positions : int32 device, the position of token n of batch b on axis a at
 *             positions[a * pos_axis_stride + b * pos_batch_stride + n]
 *             (pos_batch_stride 0: the same for every batch)
 *   inv_freq : double [sum of sections] device, finite, radians per position
 *   sections : host array of num_sections (1..4) pair counts, each >= 1: the
 *             first sections[0] pairs turn by axis 0, the next by axis 1, ...
 *             Their sum is the number of rotated pairs: at most d / 2, a multiple
 *             of 8 (ATTN_ERR_UNSUPPORTED otherwise).
 *   interleaved : 0: pair i is elements (i, i + pairs); otherwise (2 i, 2 i + 1)
 *   d : 64 or 128;  eps : finite, >= 0;  B, Hq, Hk, N >= 1, products B*N*H < 2^31 - 512
 * Asynchronous on `stream`; no workspace.
 */
int attn_qk_norm_rope(const void* Q, const int64_t* q_strides, const void* K, const int64_t* k_strides,
                      const void* q_weight, const void* k_weight, const int32_t* positions, int64_t pos_axis_stride,
                      int64_t pos_batch_stride, const double* inv_freq, const int* sections, int num_sections,
                      void* Qout, const int64_t* qo_strides, void* Kout, const int64_t* ko_strides, int B, int Hq,
                      int Hk, int N, int d, float eps, int interleaved, cudaStream_t stream);

/*
 * attn_qk_norm_rope_bwd - gradients of attn_qk_norm_rope for upstream gradients
 * dQout, dKout of its outputs (attn_bwd's dQ and dK).  With u the upstream row
 * turned back by the angles and h = x / sqrt(mean x^2 + eps):
 *     dx = (u w - h mean_j(u_j w_j h_j)) / sqrt(mean x^2 + eps),
 *     dweight_j = sum over batch, head and token of u_j h_j;
 * without a weight dx = u, and Q (or K) is not read and may be NULL.
 *   dQout, Q, dQ : bf16 [B, Hq, N, d] device views, and dKout, K, dK likewise:
 *             layouts, strides and alignment as above.  dQ may be dQout or Q in
 *             place (its address and strides).  An expanded input's gradient is that of
 *             the expanded view: summing it is the caller's.
 *   dq_weight, dk_weight : fp32 [d] device (written), NULL exactly where the weight is
 *             NULL (ATTN_ERR_INVALID_ARG otherwise).  Summed in fp32 in a fixed
 *             order: the same call gives the same bits.
 *   workspace : device buffer of at least attn_qk_norm_rope_bwd_workspace_bytes(),
 *             16-byte aligned, owned by the caller, not used by other work while
 *             this call runs; may be NULL when neither weight is given
 * Other arguments and errors as attn_qk_norm_rope.  Asynchronous on `stream`.
 */
int attn_qk_norm_rope_bwd(const void* dQout, const int64_t* dqo_strides, const void* dKout, const int64_t* dko_strides,
                          const void* Q, const int64_t* q_strides, const void* K, const int64_t* k_strides,
                          const void* q_weight, const void* k_weight, const int32_t* positions, int64_t pos_axis_stride,
                          int64_t pos_batch_stride, const double* inv_freq, const int* sections, int num_sections,
                          void* dQ, const int64_t* dq_strides, void* dK, const int64_t* dk_strides, float* dq_weight,
                          float* dk_weight, int B, int Hq, int Hk, int N, int d, float eps, int interleaved,
                          void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Device bytes attn_qk_norm_rope_bwd needs as workspace on the current device:
 * an fp32 row of d per CTA; 0 for d other than 64 or 128, or without a device. */
size_t attn_qk_norm_rope_bwd_workspace_bytes(int d);

/*
 * attn_fwd_prefix - attention of a batch of requests that share a long prefix
 * (one prompt or document and many continuations): T new tokens of each of R
 * requests against the prefix's keys and values, stored once for all, and the
 * request's own,
 *     O = softmax(scale * q [Kp; Ko_r]^T) [Vp; Vo_r]  and its log-sum-exp.
 * The rows of all requests and of the Hq / Hk query heads that share a key head
 * form one tall matrix against the prefix (the tall-and-skinny product of the
 * AttenIO abstract), so the prefix is read once, not once per request.  Both key ranges run as the
 * streaming pass of attn_fwd in pieces, merged like attn_fwd_split's segments.
 *   Q, O    : bf16 [R, Hq, T, d] device views; Hq a multiple of Hk, query head h
 *             reads key head h / (Hq / Hk)
 *   Kp, Vp  : bf16 [Hk, P, d] device views; P = 0: no prefix (then they may be NULL)
 *   Ko, Vo  : bf16 [R, Hk, C, d] device views, caches of capacity C; C = 0: no own
 *             keys (then they, and own_lens where no request is padding, may be NULL).
 *             P and C are not both 0.
 *   own_lens: int32 [R] device: the request's own keys, its T new tokens (the
 *             last of them) among them; more than C counts as C.  0: none: the rows see
 *             the prefix alone (without one: O = 0, LSE = -inf).  Negative: the
 *             request is padding and its rows of O and LSE stay as they were.
 *             Read on the device, so a captured graph may be replayed with other lengths.
 *   Masking : every token sees the whole prefix; token t of T sees the own keys
 *             j < own_lens - (T - 1 - t).  Cache rows at and past own_lens are not
 *             used and may hold anything, NaN included.  A NaN or infinity in a new token's K
 *             reaches only the tokens that see it; in its V it reaches every token of that
 *             request (its weight for the others is 0, and 0 times it is a NaN).
 *   LSE     : fp32 [R, Hq, T] device, contiguous (natural log)
 *   *_strides : host arrays in elements, outermost axis first, d contiguous (Q,
 *             O: request, head, token; Kp, Vp: head, key; Ko, Vo: request, head, key);
 *             NULL: contiguous.  Positive multiples of 8 for axes longer than 1, and
 *             stride times extent at most 2^39.
 *   d       : 64 or 128;  scale : any finite value;  R, Hq, Hk, T >= 1; R*Hq*T, P and C below
 *             2^31 - 512, and less than 2^30 tiles of work (Hk * P / 128; R * Hk * C / 16)
 *   workspace : device buffer of at least attn_fwd_prefix_workspace_bytes(), 16-byte
 *             aligned, owned by the caller, not used by other work while this call runs
 *             (calls that may overlap, captured graphs among them, need one each)
 * Arithmetic as attn_fwd (fp32 scores and sums, P rounded to bf16); pieces are
 * kept in fp32, O is rounded once.  The cut into pieces depends on the own
 * lengths, so bits may differ between batches, not between equal calls.
 * Two or three launches on `stream`.  Kernel-side timeouts: attn_last_device_error().
 */
int attn_fwd_prefix(const void* Q, const int64_t* q_strides, const void* Kp, const int64_t* kp_strides, const void* Vp,
                    const int64_t* vp_strides, const void* Ko, const int64_t* ko_strides, const void* Vo,
                    const int64_t* vo_strides, const int32_t* own_lens, void* O, const int64_t* o_strides, float* LSE,
                    int R, int Hq, int Hk, int T, int P, int C, int d, float scale, void* workspace,
                    size_t workspace_bytes, cudaStream_t stream);

/* Device bytes attn_fwd_prefix needs as workspace on the current device (its
 * partial rows); 0 for an invalid shape or without a device. */
size_t attn_fwd_prefix_workspace_bytes(int R, int Hq, int Hk, int T, int P, int C, int d);

/*
 * attn_fwd_packed - attention of sequences of different lengths whose tokens
 * follow one another in Q, K and V, with grouped heads:
 *     O = softmax(scale * Q K^T + mask) V  and its log-sum-exp,
 * each query over the keys of its own sequence.  The heads of a group are rows
 * of one matrix against their key head, and the work of all sequences is cut
 * into even shares for the SMs (the tall-and-skinny products and their balance
 * are the AttenIO abstract's), whatever the lengths are.
 *   Q, O    : bf16 [Hq, Nq, d] device views; Hq a multiple of Hk (at most 64 Hk, ATTN_ERR_UNSUPPORTED
 *             beyond), query head h reads key head h / (Hq / Hk)
 *   K, V    : bf16 [Hk, Nk, d] device views
 *   q_starts, k_starts : int32 [R + 1] device: sequence s has the queries
 *             q_starts[s] .. q_starts[s + 1] - 1 and the keys k_starts[s] .. k_starts[s + 1] - 1,
 *             either of which may be none.  The two may be the same array.  Read on the device, so a
 *             captured graph may be replayed with other lengths.  Offsets outside the tensors are
 *             clipped to them, and a sequence whose end is before its start is empty (so zeros behind the
 *             last sequence pad a batch); sequences must not overlap in Q (their rows would be written twice).
 *   causal  : not 0: query t of a sequence's n sees the keys j <= t + m - n of its m, so that the
 *             last query sees all of them; with more queries than keys the first see none
 *   A row that sees no key is O = 0, LSE = -inf.  Rows of tokens that are in no sequence stay
 *   as they were.  K and V rows of other sequences are not used, whatever they hold; a NaN or
 *   infinity in V reaches every row of its own sequence that is computed in the same tile of 128 keys.
 *   LSE     : fp32 [Hq, Nq] device, contiguous (natural log)
 *   *_strides : host arrays of two strides in elements (head, token), d contiguous; NULL:
 *             contiguous.  Positive multiples of 8 for axes longer than 1, and stride times
 *             extent at most 2^39.
 *   R, Nq, Nk >= 1; Hq * Nq and Hk * Nk below 2^31 - 512;  d : 64 or 128;  scale : any finite value
 *   workspace : device buffer of at least attn_fwd_packed_workspace_bytes(), 16-byte
 *             aligned, owned by the caller, not used by other work while this call runs
 *             (calls that may overlap, captured graphs among them, need one each)
 * Arithmetic as attn_fwd (fp32 scores and sums, P rounded to bf16); pieces of a row's
 * keys are kept in fp32, O is rounded once.  The cut into pieces depends on the
 * lengths of all sequences, so bits may differ between batches, not between equal calls.
 * One or two launches on `stream`, the first behind all work before it there.  Kernel-side timeouts: attn_last_device_error().
 */
int attn_fwd_packed(const void* Q, const int64_t* q_strides, const void* K, const int64_t* k_strides, const void* V,
                    const int64_t* v_strides, const int32_t* q_starts, const int32_t* k_starts, void* O,
                    const int64_t* o_strides, float* LSE, int R, int Nq, int Nk, int Hq, int Hk, int d, int causal,
                    float scale, void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Device bytes attn_fwd_packed needs as workspace on the current device (its
 * partial rows); 0 for an invalid shape or without a device.  Room for the most that any lengths can cut: next to
 * nothing up to 640 keys in all, else up to 40 MB at d = 128 (20 MB at 64), for each 128 MB of K and V again, at most 8 times. */
size_t attn_fwd_packed_workspace_bytes(int R, int Nq, int Nk, int Hq, int Hk, int d);

/*
 * attn_bwd_packed - gradients of attn_fwd_packed for an upstream gradient dO of
 * O (attn_bwd's, each query against the keys of its own sequence), with P recomputed from
 * the forward's LSE.  dK and dV are those of the key heads: summed over the query heads of a group.
 *   Q, K, V, O, dO, dQ, dK, dV : bf16 device views shaped as in attn_fwd_packed (dO and dQ like
 *             Q, dK like K, dV like V), strides as there; O and LSE as attn_fwd_packed wrote them
 *   LSE     : fp32 [Hq, Nq] device, contiguous
 *   q_starts, k_starts : as there; the sequences must not overlap in K either
 *   Rows of dQ, and of dK and dV, of tokens that are in no sequence stay as they were; keys that no query sees
 *   get 0, and so does a query that sees no key.  Rows of other sequences are not used, whatever
 *   they hold; a NaN or infinity reaches the gradients of its own sequence, also where a mask hides it.
 *   workspace : device buffer of at least attn_bwd_packed_workspace_bytes(), 16-byte
 *             aligned, owned by the caller, not used by other work while this call runs
 * Other arguments and errors as attn_fwd_packed.  dQ is summed over the key tiles in fp32 in the order in
 * which they are done, so its last bits may differ between equal calls; dK and dV do not.
 * No gradient flows into LSE.  Three launches on `stream`.  Kernel-side timeouts: attn_last_device_error().
 */
int attn_bwd_packed(const void* Q, const int64_t* q_strides, const void* K, const int64_t* k_strides, const void* V,
                    const int64_t* v_strides, const void* O, const int64_t* o_strides, const float* LSE, const void* dO,
                    const int64_t* do_strides, const int32_t* q_starts, const int32_t* k_starts, void* dQ,
                    const int64_t* dq_strides, void* dK, const int64_t* dk_strides, void* dV, const int64_t* dv_strides,
                    int R, int Nq, int Nk, int Hq, int Hk, int d, int causal, float scale, void* workspace,
                    size_t workspace_bytes, cudaStream_t stream);

/* Device bytes attn_bwd_packed needs as workspace on the current device (the
 * sums of dQ, a number per row, pieces of dK and dV); 0 for an invalid shape or
 * without a device.  4 (d + 1) bytes for each row of Q, and, for more tokens than 8 blocks of 64 / (Hq / Hk), room for the most
 * that any lengths can cut: 40 MB at d = 128 (20 MB at 64), for each 150 MB of Q, dO and the sums again, at most 32 times. */
size_t attn_bwd_packed_workspace_bytes(int R, int Nq, int Nk, int Hq, int Hk, int d);

/*
 * attn_fwd_tree - attention of T new tokens of each of R requests over keys and
 * values in the pages of a cache: single tokens, a run of tokens, or a tree of
 * drafted tokens that are checked at once.  The request's new tokens are the
 * last T of its keys; every new token sees the keys before them, and of the new
 * ones those that its row of tree_mask names.  Computed as attn_fwd_packed.
 *   Q, O    : bf16 [R, Hq, T, d] device views; Hq a multiple of Hk, as above
 *   Kc, Vc  : bf16 [pages, Hk, page_size, d] device views; page_size a power of two
 *             from 16 to 1024 (ATTN_ERR_UNSUPPORTED otherwise)
 *   page_table : int32 [R][table_pages] device, rows table_stride apart: the pages of a
 *             request's keys in order.  Only those of its keys are read; an entry
 *             that is no page of the cache reads as zeros.
 *   lens    : int32 [R] device: the request's keys, its T new tokens (the last of them)
 *             among them; more than table_pages * page_size counts as that.  0: none:
 *             O = 0, LSE = -inf.  Negative: the request is padding and its rows stay as
 *             they were.  Of a len below T the new tokens are the last of T: those before are missing.
 *   tree_mask : int32 [R, T, ceil(T / 32)] device, contiguous, or NULL: new token t sees
 *             new token j where bit j % 32 of word j / 32 of its row is set (its own bit is
 *             not implied; bits past T do not count).  NULL: it sees those up to itself.
 *             Read on the device, as lens and page_table: a captured graph may be replayed with others.
 *   A row that sees no key is O = 0, LSE = -inf.  Cache rows that are not a request's
 *   keys may hold anything, NaN included.  A NaN or infinity in a new token's K reaches
 *   only the tokens that see it; in its V it reaches every new token of that request.
 *   LSE     : fp32 [R, Hq, T] device, contiguous (natural log)
 *   *_strides : host arrays of three strides in elements (Q, O: request, head, token;
 *             Kc, Vc: page, head, key), as above;  table_stride : elements, >= 0
 *   d       : 64 or 128;  scale : any finite value;  R, T, pages, table_pages >= 1; R * Hq * T,
 *             pages and table_pages * page_size below 2^31 - 512
 *   workspace : attn_fwd_tree_workspace_bytes(), as above
 * One or two launches on `stream`.  Kernel-side timeouts: attn_last_device_error().
 */
int attn_fwd_tree(const void* Q, const int64_t* q_strides, const void* Kc, const int64_t* k_strides, const void* Vc,
                  const int64_t* v_strides, const int32_t* page_table, int64_t table_stride, const int32_t* lens,
                  const int32_t* tree_mask, void* O, const int64_t* o_strides, float* LSE, int R, int Hq, int Hk, int T,
                  int pages, int page_size, int table_pages, int d, float scale, void* workspace, size_t workspace_bytes,
                  cudaStream_t stream);

/* Device bytes attn_fwd_tree needs as workspace on the current device (up to 40 MB at d = 128, 20 MB at 64, whatever
 * the cache holds); 0 for an invalid shape or without a device. */
size_t attn_fwd_tree_workspace_bytes(int R, int Hq, int Hk, int T, int d);

#ifdef __cplusplus
}
#endif

#endif /* EXACT_ATTN_H */
