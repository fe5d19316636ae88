// Log probabilities of materialised logits: a given token's, the row's
// log-sum-exp and entropy, the best alternatives; and their gradient.
//
// With m = max l, S = sum exp((l - m)/T) and A = sum (l - m)/T exp((l - m)/T)
// over the unmasked ids of a row:  lse = m/T + ln S,  log p_i = (l_i - m)/T -
// ln S,  entropy = ln S - A/S.
#include "fs_vocab.h"

namespace fs {

constexpr int kLpThreads = 256;

template <int DT>
__device__ __forceinline__ float row_logit(const void* row, const uint32_t* allow_row, int i) {
    const float l = (float)static_cast<const typename Elem<DT>::type*>(row)[i];
    return allowed(allow_row, i) ? clean_logit(l) : -INFINITY;
}

template <typename F, typename V>
__device__ V block_reduce(V v, V* slot, F op) {
    __syncthreads();
    slot[threadIdx.x] = v;
    __syncthreads();
    for (int s = kLpThreads / 2; s >= 1; s >>= 1) {
        if (threadIdx.x < s) slot[threadIdx.x] = op(slot[threadIdx.x], slot[threadIdx.x + s]);
        __syncthreads();
    }
    return slot[0];
}

template <int DT>
__global__ __launch_bounds__(kLpThreads) void logprobs_kernel(LogprobsArgs a) {
    __shared__ float fslot[kLpThreads];
    __shared__ int islot[kLpThreads];
    __shared__ uint64_t kslot[kLpThreads];
    const int Vv = min((int64_t)a.V, max((int64_t)0, (int64_t)a.n_valid - a.v_offset));
    auto add = [](float x, float y) { return x + y; };
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const void* row =
            static_cast<const char*>(a.logits) + (size_t)b * a.ld * sizeof(typename Elem<DT>::type);
        const uint32_t* allow_row = a.allow ? a.allow + (size_t)b * ((a.V + 31) >> 5) : nullptr;
        const float T = row_temp(a.temp, b, a.flags);
        float m = -INFINITY;
        for (int i = threadIdx.x; i < Vv; i += kLpThreads)
            m = fmaxf(m, row_logit<DT>(row, allow_row, i));
        m = block_reduce(m, fslot, [](float x, float y) { return fmaxf(x, y); });
        const int tok = a.token ? a.token[b] - a.v_offset : -1;
        const float lt = tok >= 0 && tok < Vv ? row_logit<DT>(row, allow_row, tok) : -INFINITY;
        float S = 0.f, A = 0.f;
        int before = 0;
        for (int i = threadIdx.x; i < Vv; i += kLpThreads) {
            const float l = row_logit<DT>(row, allow_row, i);
            if (!(l > -INFINITY)) continue;
            const float x = (l - m) / T;
            const float e = __expf(x);
            S += e;
            A += e > 0.f ? x * e : 0.f;
            before += l > lt || (l == lt && i < tok);
        }
        S = block_reduce(S, fslot, add);
        A = block_reduce(A, fslot, add);
        before = block_reduce(before, islot, [](int x, int y) { return x + y; });
        const bool any = m > -INFINITY;
        const float logS = logf(S);
        if (threadIdx.x == 0) {
            const bool has = lt > -INFINITY;
            if (a.logprob) a.logprob[b] = has ? (lt - m) / T - logS : -INFINITY;
            if (a.rank) a.rank[b] = has ? before + 1 : 0;
            if (a.lse) a.lse[b] = any ? m / T + logS : -INFINITY;
            if (a.entropy) a.entropy[b] = any ? logS - A / S : 0.f;
        }
        uint64_t last = ~0ull;
        for (int j = 0; j < a.n_top; ++j) {
            uint64_t best = 0;
            for (int i = threadIdx.x; i < Vv; i += kLpThreads) {
                const float l = row_logit<DT>(row, allow_row, i);
                const uint64_t k = l > -INFINITY ? pack_key(l, i) : 0;
                if (k < last) best = key_max(best, k);
            }
            best = block_reduce(best, kslot, [](uint64_t x, uint64_t y) { return key_max(x, y); });
            last = best;
            if (threadIdx.x == 0) {
                const size_t o = (size_t)b * a.n_top + j;
                a.top_idx[o] = best ? key_index(best) + a.v_offset : -1;
                a.top_logprob[o] = best ? (key_score(best) - m) / T - logS : -INFINITY;
            }
        }
    }
}

// dl_i = 1/T [ p_i (g_lse - g_lp - sum_j g_top_j - g_H (ln p_i + H))
//              + [i = token] g_lp + sum_j [i = top_j] g_top_j ],  ln p_i = x_i - lse.
template <int DT>
__global__ __launch_bounds__(kLpThreads) void logprobs_grad_kernel(LogprobsGradArgs a) {
    typedef typename Elem<DT>::type E;
    const int Vv = min((int64_t)a.V, max((int64_t)0, (int64_t)a.n_valid - a.v_offset));
    for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
        const E* row = static_cast<const E*>(a.logits) + (size_t)b * a.ld;
        E* out = static_cast<E*>(a.grad) + (size_t)b * a.ld_grad;
        const uint32_t* allow_row = a.allow ? a.allow + (size_t)b * ((a.V + 31) >> 5) : nullptr;
        const float T = row_temp(a.temp, b, a.flags);
        const float lse = a.lse[b];
        const float glp = a.g_logprob ? a.g_logprob[b] : 0.f;
        const float gH = a.g_entropy ? a.g_entropy[b] : 0.f;
        const float H = a.g_entropy ? a.entropy[b] : 0.f;
        const int tok_id = a.g_logprob ? a.token[b] : -1;
        const int tok = tok_id >= 0 ? tok_id - a.v_offset : -1;
        float c = (a.g_lse ? a.g_lse[b] : 0.f) - (tok_id >= 0 ? glp : 0.f);
        for (int j = 0; a.g_top && j < a.n_top; ++j)
            if (a.top_idx[(size_t)b * a.n_top + j] >= 0) c -= a.g_top[(size_t)b * a.n_top + j];
        for (int i = blockIdx.x * kLpThreads + threadIdx.x; i < a.V; i += gridDim.x * kLpThreads) {
            const float l = i < Vv ? row_logit<DT>(row, allow_row, i) : -INFINITY;
            float g = 0.f;
            if (l > -INFINITY && fabsf(lse) < INFINITY) {
                const float lp = l / T - lse;
                const float p = __expf(lp);
                g = p > 0.f ? p * (c - gH * (lp + H)) : 0.f;
                if (i == tok) g += glp;
                for (int j = 0; a.g_top && j < a.n_top; ++j)
                    if (a.top_idx[(size_t)b * a.n_top + j] - a.v_offset == i)
                        g += a.g_top[(size_t)b * a.n_top + j];
                g /= T;
            }
            out[i] = (E)g;
        }
    }
}

hipError_t launch_logprobs(const LogprobsArgs& a, void* ws, hipStream_t stream) {
    (void)ws;
    const dim3 grid(a.B);
    if (a.dtype == FS_F32)
        hipLaunchKernelGGL(logprobs_kernel<FS_F32>, grid, dim3(kLpThreads), 0, stream, a);
    else if (a.dtype == FS_BF16)
        hipLaunchKernelGGL(logprobs_kernel<FS_BF16>, grid, dim3(kLpThreads), 0, stream, a);
    else
        hipLaunchKernelGGL(logprobs_kernel<FS_F16>, grid, dim3(kLpThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_logprobs_grad(const LogprobsGradArgs& a, hipStream_t stream) {
    const dim3 grid((a.V + 4095) / 4096, a.B < kMaxGridY ? a.B : kMaxGridY);
    if (a.dtype == FS_F32)
        hipLaunchKernelGGL(logprobs_grad_kernel<FS_F32>, grid, dim3(kLpThreads), 0, stream, a);
    else if (a.dtype == FS_BF16)
        hipLaunchKernelGGL(logprobs_grad_kernel<FS_BF16>, grid, dim3(kLpThreads), 0, stream, a);
    else
        hipLaunchKernelGGL(logprobs_grad_kernel<FS_F16>, grid, dim3(kLpThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace fs
