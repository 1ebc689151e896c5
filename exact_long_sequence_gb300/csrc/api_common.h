// Host-side pieces shared by the library's entry points (forward, backward):
// per-device state, status bookkeeping, argument checks and TMA descriptors.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/exact_attn.h"

namespace elsattn {

constexpr int kMaxDevices = 64;
constexpr uint64_t kDefaultTimeoutNs = 4000000000ull;  // 4 s for any single wait

// Sizes that kernels round up to whole tiles, row blocks (of at most 256) and steps in 32 bits stay below this.
constexpr long long kRoundedSizeLimit = (1LL << 31) - 512;

struct DeviceState {
    bool ready = false;
    int num_sms = 0;
    int cc_major = 0, cc_minor = 0;
    uint32_t* error_word = nullptr;  // 256-byte device block, first word = error code
    bool smem_configured[2][2][2] = {};                                   // forward <d == 128><causal><dynamic schedule>
    bool bwd_smem_configured[2][2] = {{false, false}, {false, false}};  // backward <d == 128><causal>
    bool prefix_smem_configured[2][2] = {};  // shared-prefix forward <own-keys kernel><d == 128>
    bool packed_smem_configured[2][2] = {};  // attention over lengths <paged><d == 128>
    bool packed_bwd_smem_configured[2] = {};  // its gradient <d == 128>
    bool ready_configured[2][8] = {};  // query / key preparation <backward><variant>
    bool fp8_smem_configured[2][2][2] = {};  // FP8 forward <causal><dynamic schedule><K/V segments>
};

// The cudaError_t of this thread's most recent ATTN_ERR_CUDA.
extern thread_local int g_last_cuda_error;

// Records `e` as this thread's last CUDA error and returns ATTN_ERR_CUDA.
int cuda_fail(cudaError_t e);

// Looks up the driver's cuTensorMapEncodeTiled once per process.
int resolve_tensor_map_encoder();

// The current device's state, set up on first use (checks for sm_103,
// resolves the tensor-map encoder, allocates the error word).
int device_state(DeviceState** out);

// A bf16 tensor viewed as [BH][N][d] (d innermost), read by TMA in boxes of
// 64 columns x box_rows rows with the 128-byte swizzle the tcgen05
// descriptors expect.  Rows past N read as zero.
int encode_rows_map(CUtensorMap* map, const void* base, int BH, int N, int d, int box_rows);

// A bf16 tensor of rank 3 to 5 with extents e (e[0] = d innermost) and byte
// strides st of the outer axes (multiples of 16), read by TMA in boxes `box`
// (box[0] = 64 columns), 128-byte swizzle.  What lies past an extent reads as zero.
int encode_bf16_map(CUtensorMap* map, const void* base, int rank, const uint64_t* e, const uint64_t* st, const uint32_t* box);

// An fp32 tensor viewed as [BH][N][d], written by TMA (reduce-add) in boxes of
// d columns x box_rows rows, unswizzled.  Rows past N are dropped.
int encode_f32_rows_map(CUtensorMap* map, void* base, int BH, int N, int d, int box_rows);

// A 3-D byte tensor (E4M3 codes) with extents {e0, e1, e2} (e0 innermost) and
// byte strides s1, s2 (multiples of 16), read by TMA in boxes of b0 x b1 with
// the 128-byte swizzle (b0 = 128).  Elements past an extent read as zero.
int encode_u8_map(CUtensorMap* map, const void* base, uint64_t e0, uint64_t e1, uint64_t e2, uint64_t s1,
                  uint64_t s2, uint32_t b0, uint32_t b1);

bool aligned16(const void* p);

// Test hook (attn_debug_arm_timeout): a one-shot time limit for the next launch that takes it; 0: not armed.
void arm_timeout(uint64_t timeout_ns);
uint64_t take_armed_timeout();

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
            if (out[i] <= 0 || out[i] >= (1LL << 39) || out[i] > (1LL << 39) / dims[i]) return ATTN_ERR_INVALID_ARG;
        }
        dense *= dims[i];
    }
    return ATTN_OK;
}

// Shared argument checks of the forward and backward entry points.
int check_args(const void* Q, const void* K, const void* V, const void* O, const void* LSE, int B, int H, int N,
               int d, float scale);

}  // namespace elsattn
