// Internal declarations of the slot router and the packed bank: launch parameter
// blocks and the launchers that the C ABI calls.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sdm {

// Between a wavefront's LDS writes and its reads of what other lanes wrote: its LDS
// accesses happen in order by themselves, so only the compiler has to keep to it.
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ------------------------------------------------------------------ route
struct RouteParams {
    const void* logits;
    const float* bias;  // NULL: no bias
    int64_t tokens;
    int keys, k;
    int score;  // SDM_SOFTMAX or SDM_SIGMOID
    int groups, kept, top;
    int normalise;
    double scale;
    uint32_t streams;  // at most that many: tokens are fewer than 2^32
    int64_t stream_slots;
    void* idx;
    void* w;
    int idx64, w_bf16;
};
hipError_t launch_route(const RouteParams& p, bool bf16, hipStream_t stream);
void launch_route_block(const RouteParams& p, bool bf16, hipStream_t stream);  // any row: a workgroup each

struct RouteBackwardParams {
    const void* logits;
    const float* bias;
    int64_t tokens;
    int keys, k;
    int score, normalise;
    double scale;
    uint32_t streams;  // at most that many: tokens are fewer than 2^32
    int64_t stream_slots;
    const void* idx;
    const void* dw;
    void* dlogits;
    int idx64, w_bf16;
};
hipError_t launch_route_backward(const RouteBackwardParams& p, bool bf16, hipStream_t stream);

// ------------------------------------------------------------------ packed bank
struct PackParams {
    uint8_t* codes;
    uint8_t* scales;
    const void* rows;
    const void* row_idx;  // NULL: row i
    const void* slots;    // NULL: slot i
    int64_t num_slots, num_rows, n;
    int hd;
    int row_bytes, scale_bytes;
    int idx64;
};
hipError_t launch_pack(const PackParams& p, bool bf16, bool mx4, hipStream_t stream);

// The two operands of a gather over a packed bank, or of a gather's weight gradient.
struct MemoryGatherParams {
    const void* bank;  // codes, or a float bank's rows
    const uint8_t* scales;
    const int32_t* chunk_valid;
    const void* idx[2];
    const void* w[2];   // weights (gather)
    float* out[2];      // (gather)
    const float* dout[2];  // (weight gradient)
    void* dw[2];           // (weight gradient)
    int width[2];
    int64_t tokens, chunk, valid, num_slots;
    int hd;
    int64_t row_bytes;
    int scale_bytes;
    int operands;
    int idx64, w_bf16;
    int out_vec;  // outputs and their rows aligned to 16 bytes (gather)
};
hipError_t launch_gather_packed(const MemoryGatherParams& p, bool mx4, hipStream_t stream);
hipError_t launch_weight_grad(const MemoryGatherParams& p, int bank_dtype, hipStream_t stream);

}  // namespace sdm
