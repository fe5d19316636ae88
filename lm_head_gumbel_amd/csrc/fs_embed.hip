// Embedding of token ids, out[n] = scale W[ids[n]], and its gradient,
// dW[v] = scale sum of g[n] over the n with ids[n] = v, in the order of n.
#include "fs_vocab.h"

namespace fs {

constexpr int kEmThreads = 256;

template <int DT>
__global__ __launch_bounds__(kEmThreads) void embed_kernel(EmbedArgs a) {
    typedef typename Elem<DT>::type E;
    for (int n = blockIdx.x; n < a.N; n += gridDim.x) {
        const int64_t j = (int64_t)a.ids[n] - a.v_offset;
        const bool in = j >= 0 && j < a.V;
        for (int k = threadIdx.x; k < a.d; k += kEmThreads)
            static_cast<E*>(a.out)[(size_t)n * a.d + k] =
                (E)(in ? a.scale * (float)static_cast<const E*>(a.W)[(size_t)j * a.d + k] : 0.f);
    }
}

// One workgroup per vocabulary row: reads every id.
template <int DT, int DO>
__global__ __launch_bounds__(kEmThreads) void embed_grad_kernel(EmbedGradArgs a) {
    typedef typename Elem<DT>::type E;
    typedef typename Elem<DO>::type O;
    __shared__ int hit[kEmThreads];
    for (int v = blockIdx.x; v < a.V; v += gridDim.x) {
        O* out = static_cast<O*>(a.dW) + (size_t)v * a.d;
        for (int k0 = 0; k0 < a.d; k0 += kEmThreads) {
            const int k = k0 + threadIdx.x;
            float sum = 0.f;
            bool any = false;
            for (int n0 = 0; n0 < a.N; n0 += kEmThreads) {
                const int n = n0 + threadIdx.x;
                hit[threadIdx.x] = n < a.N && (int64_t)a.ids[n] - a.v_offset == v;
                if (__syncthreads_or(hit[threadIdx.x])) {
                    any = true;
                    for (int i = 0; i < kEmThreads && n0 + i < a.N; ++i)
                        if (hit[i] && k < a.d)
                            sum += (float)static_cast<const E*>(a.g)[(size_t)(n0 + i) * a.d + k];
                }
                __syncthreads();
            }
            if (k < a.d && (any || !a.accumulate))
                out[k] = (O)((a.accumulate ? (float)out[k] : 0.f) + a.scale * sum);
        }
    }
}

hipError_t launch_embed(const EmbedArgs& a, hipStream_t stream) {
    const dim3 grid(a.N);
    if (a.dtype == FS_F32)
        hipLaunchKernelGGL(embed_kernel<FS_F32>, grid, dim3(kEmThreads), 0, stream, a);
    else if (a.dtype == FS_BF16)
        hipLaunchKernelGGL(embed_kernel<FS_BF16>, grid, dim3(kEmThreads), 0, stream, a);
    else
        hipLaunchKernelGGL(embed_kernel<FS_F16>, grid, dim3(kEmThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_embed_grad(const EmbedGradArgs& a, void* ws, hipStream_t stream) {
    (void)ws;
    const dim3 grid(a.V < (1 << 20) ? a.V : 1 << 20);
#define FS_EG(DT_, DO_)                                                                       \
    if (a.dtype == DT_ && a.dw_dtype == DO_) {                                                \
        hipLaunchKernelGGL((embed_grad_kernel<DT_, DO_>), grid, dim3(kEmThreads), 0, stream, a); \
        return hipGetLastError();                                                             \
    }
    FS_EG(FS_F32, FS_F32)
    FS_EG(FS_BF16, FS_F32)
    FS_EG(FS_BF16, FS_BF16)
    FS_EG(FS_F16, FS_F32)
    FS_EG(FS_F16, FS_F16)
#undef FS_EG
    return hipErrorInvalidValue;
}

}  // namespace fs
