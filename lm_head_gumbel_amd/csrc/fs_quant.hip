// Logits of a W held in 4 bits with a scale (and a zero point) per group of
// consecutive k.
#include "fs_vocab.h"

namespace fs {

__device__ __forceinline__ float quant_scale(const void* s, int dtype, size_t i) {
    if (dtype == FS_F32) return static_cast<const float*>(s)[i];
    if (dtype == FS_BF16) return (float)static_cast<const __bf16*>(s)[i];
    return (float)static_cast<const _Float16*>(s)[i];
}

// One wave per (W row, batch row).
__global__ __launch_bounds__(256) void quant_kernel(QuantArgs a) {
    const int lane = threadIdx.x & 63;
    const int j = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (j >= a.V) return;
    const int ng = a.d / a.group;
    const uint8_t* q = a.q + (size_t)j * (a.d / 2);
    for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
        const __bf16* h = reinterpret_cast<const __bf16*>(a.H) + (size_t)b * a.d;
        float acc = 0.f;
        for (int k = lane * 2; k < a.d; k += 128) {
            const size_t g = (size_t)j * ng + k / a.group;
            const float s = quant_scale(a.scale, a.scale_dtype, g);
            const int z = a.zero ? a.zero[g] : 8;
            const uint8_t v = q[k / 2];
            acc = fmaf(s * (float)((int)(v & 15) - z), (float)h[k], acc);
            acc = fmaf(s * (float)((int)(v >> 4) - z), (float)h[k + 1], acc);
        }
        for (int m = 32; m >= 1; m >>= 1) acc += __shfl_xor(acc, m, 64);
        if (lane == 0) a.logits[(size_t)b * a.V + j] = acc;
    }
}

hipError_t launch_quant(const QuantArgs& a, int cus, hipStream_t stream) {
    (void)cus;
    hipLaunchKernelGGL(quant_kernel, dim3((a.V + 3) / 4, a.B < kMaxGridY ? a.B : kMaxGridY),
                       dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace fs
