// Interfaces of the vocabulary operators beside the sampler: logits of a
// 4-bit W (fs_quant.hip), log probabilities and their gradient
// (fs_logprobs.hip), the embedding and its gradient (fs_embed.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fs.h"
#include "fs_device.h"
#include "fs_plan.h"

namespace fs {

// Element types (FS_F32, FS_BF16, FS_F16): arithmetic is FP32, a store rounds
// to nearest, ties to even.
template <int DT>
struct Elem {
    typedef float type;
};
template <>
struct Elem<FS_BF16> {
    typedef __bf16 type;
};
template <>
struct Elem<FS_F16> {
    typedef _Float16 type;
};

struct QuantArgs {
    const uint16_t* H;     // [B, d] bf16
    const uint8_t* q;      // [V, d / 2]
    const void* scale;     // [V, d / group]
    const uint8_t* zero;   // [V, d / group] or null (8)
    float* logits;         // [B, V]
    int B, d, V, group, scale_dtype;
};
hipError_t launch_quant(const QuantArgs& a, int cus, hipStream_t stream);

struct LogprobsArgs {
    const void* logits;   // [B] rows of V elements, ld apart
    int dtype;
    int64_t ld;
    const float* temp;
    const uint32_t* allow;
    const int32_t* token;
    int B, V, n_valid, v_offset, n_top;
    uint32_t flags;
    float* logprob;
    int32_t* rank;
    float* lse;
    float* entropy;
    int32_t* top_idx;
    float* top_logprob;
};
// Workspace of a call (0: none), the same cus as the launch.
size_t logprobs_ws_bytes(int B, int V, int n_top, int cus);
hipError_t launch_logprobs(const LogprobsArgs& a, void* ws, int cus, hipStream_t stream);

struct LogprobsGradArgs {
    const void* logits;
    void* grad;
    int dtype;
    int64_t ld, ld_grad;
    const float* temp;
    const uint32_t* allow;
    const int32_t* token;
    const int32_t* top_idx;
    const float* lse;
    const float* entropy;
    const float* g_logprob;
    const float* g_lse;
    const float* g_entropy;
    const float* g_top;
    int B, V, n_valid, v_offset, n_top;
    uint32_t flags;
};
hipError_t launch_logprobs_grad(const LogprobsGradArgs& a, hipStream_t stream);

struct EmbedArgs {
    const int32_t* ids;   // [N]
    const void* W;        // [V, d]
    void* out;            // [N, d]
    int N, d, V, v_offset, dtype;
    float scale;
};
hipError_t launch_embed(const EmbedArgs& a, hipStream_t stream);

struct EmbedGradArgs {
    const int32_t* ids;   // [N]
    const void* g;        // [N, d]
    void* dW;             // [V, d]
    int N, d, V, v_offset, dtype, dw_dtype;
    float scale;
    int accumulate;
};
size_t embed_grad_ws_bytes(int N, int d);
hipError_t launch_embed_grad(const EmbedGradArgs& a, void* ws, hipStream_t stream);

// A row's temperature: 1 where it is greedy, as the shared definitions say.
__device__ __forceinline__ float row_temp(const float* temp, int b, uint32_t flags) {
    const float T = temp ? temp[b] : 1.f;
    return (flags & kFlagNoNoise) || !(T > 0.f) ? 1.f : T;
}

__device__ __forceinline__ bool allowed(const uint32_t* allow_row, int i) {
    return !allow_row || ((allow_row[i >> 5] >> (i & 31)) & 1u);
}

}  // namespace fs
