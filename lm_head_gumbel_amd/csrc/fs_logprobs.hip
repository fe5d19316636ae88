// Log probabilities of materialised logits: a given token's and its rank, the
// row's log-sum-exp and entropy, the best alternatives; and their gradient.
//
// With m = max l, x_i = (l_i - m) / T, S = sum e^{x_i} and A = sum x_i e^{x_i}
// over the unmasked ids of a row:  lse = m / T + ln S,  ln p_i = x_i - ln S,
// entropy = ln S - A / S.  (m, S, A) of disjoint slices join: with M the
// larger m and w = e^{(m - M) / T}, S adds w S and A adds w (A + (m - M) / T S).
//
// Bound by the one read of the logits.  A workgroup takes a slice of a row
// into registers (E elements a thread, all loads issued before the first
// use), so the slice's maximum is known before the first exponential and no
// running sum is ever rescaled; a second kernel joins the slices of a row.
// MI355X: 2048 x 128256 bf16 in 142 us, 3.7 TB/s, where the exponential of
// every element (a quarter-rate instruction) bounds it; 4096 x 32000 FP32 in 89
// us, 5.9 TB/s; 1 x 151936 FP32 with 20 alternatives in 14 us, all latency.
#include <algorithm>
#include <type_traits>

#include "fs_vocab.h"

namespace fs {

namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWaves = kLpThreads / 64;
constexpr int kLpShort = 8;    // elements per thread of a short slice
constexpr int kLpLong = 32;    // and of a long one
constexpr int kJoinEntries = 2048;   // alternatives of a row's slices that the join keeps in LDS
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
constexpr float kMaxFloat = 3.402823466e38f;
constexpr float kFloor = -1e30f;   // exponents: e^{-inf} without inf * 0

// 16 bytes of elements as they lie in memory, four 32-bit words.
template <int DT>
struct Vec {
    typedef typename Elem<DT>::type E;
    static constexpr int kN = 16 / (int)sizeof(E);   // elements
    uint32_t w[4];
    // element e in FP32
    __device__ __forceinline__ float at(int e) const {
        if constexpr (DT == FS_F32) return __uint_as_float(w[e]);
        const uint32_t h = e % 2 ? w[e / 2] >> 16 : w[e / 2];
        return DT == FS_BF16 ? __uint_as_float(h << 16)
                             : (float)__builtin_bit_cast(_Float16, (uint16_t)h);
    }
};
// -inf in both halves (or the whole) of a word.
template <int DT>
constexpr uint32_t kMinusInf = DT == FS_F32 ? 0xFF800000u : DT == FS_BF16 ? 0xFF80FF80u : 0xFC00FC00u;

// Ids of the row that can be unmasked.
__device__ __forceinline__ int valid_ids(int V, int n_valid, int v_offset) {
    return (int)min((int64_t)V, max((int64_t)0, (int64_t)n_valid - v_offset));
}

// FP32 logit: NaN -> -inf, +inf -> the largest finite value.
__device__ __forceinline__ float clean(float l) {
    return fminf(l == l ? l : -INFINITY, kMaxFloat);
}

// Bit o of the result: id i + o is allowed (o < n <= 8; i + n <= V).
__device__ __forceinline__ uint32_t allow_bits(const uint32_t* row, int i, int n) {
    const uint32_t lo = row[i >> 5], hi = row[(i + n - 1) >> 5];
    const int sh = i & 31;
    return sh + n > 32 ? (lo >> sh) | (hi << (32 - sh)) : lo >> sh;
}

// A wave's chunk of 64 kN consecutive ids of a row: whole inside the row, a
// lane holds kN consecutive ids from one 16-byte load (at any alignment of
// the row to its element size); where the row ends inside, lane l holds ids
// l, l + 64, ..  Everything here but the lane is the same for the whole wave.
template <int DT>
struct Chunk {
    static constexpr int kN = Vec<DT>::kN;
    int first, lane0, step;   // id of element e: first + lane0 + e * step
    bool whole;
    __device__ __forceinline__ Chunk(int first_, int n, int lane) : first(first_) {
        whole = first + 64 * kN <= n;
        lane0 = whole ? lane * kN : lane;
        step = whole ? 1 : 64;
    }
    __device__ __forceinline__ int id(int e) const { return first + lane0 + e * step; }
};
// Its elements (-inf past the end; STREAM: read past the caches), and bit e of
// `bits`: element e is allowed.
template <int DT, bool MASKED, bool STREAM>
__device__ __forceinline__ void load_chunk(const Chunk<DT>& c,
                                           const typename Elem<DT>::type* row,
                                           const uint32_t* allow_row, int n,
                                           Vec<DT>& v, uint32_t& bits) {
    constexpr int N = Vec<DT>::kN;
    bits = ~0u;
    if (c.whole) {
        typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));
        const u32x4* p = reinterpret_cast<const u32x4*>(row + c.id(0));
        const u32x4 w = STREAM ? __builtin_nontemporal_load(p) : *p;
        __builtin_memcpy(v.w, &w, 16);
        if constexpr (MASKED) bits = allow_bits(allow_row, c.id(0), N);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v.w[i] = kMinusInf<DT>;
        if (c.first >= n) return;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int id = c.id(e);
            if (id < n) {
                const typename Elem<DT>::type one = row[id];
                if constexpr (DT == FS_F32)
                    v.w[e] = __builtin_bit_cast(uint32_t, one);
                else
                    v.w[e / 2] = (v.w[e / 2] & (e % 2 ? 0xFFFFu : 0xFFFF0000u)) |
                                 ((uint32_t)__builtin_bit_cast(uint16_t, one) << (e % 2 * 16));
                if constexpr (MASKED)
                    if (!((allow_row[id >> 5] >> (id & 31)) & 1u)) bits &= ~(1u << e);
            }
        }
    }
}

// Reductions of a wave in its vector registers (data-parallel primitives: a
// row of 16 lanes in four steps, the rows in two), the same in every lane.
template <int CTRL, int ROWS, typename T>
__device__ __forceinline__ T lanes_from(T v, T identity) {
    static_assert(sizeof(T) == 4, "one register");
    return __builtin_bit_cast(
        T, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, identity), __builtin_bit_cast(int, v),
                                       CTRL, ROWS, 0xF, false));
}
template <typename T, typename F>
__device__ __forceinline__ T wave_reduce(T v, T identity, F op) {
    v = op(v, lanes_from<0x111, 0xF>(v, identity));   // row_shr 1, 2, 4, 8
    v = op(v, lanes_from<0x112, 0xF>(v, identity));
    v = op(v, lanes_from<0x114, 0xF>(v, identity));
    v = op(v, lanes_from<0x118, 0xF>(v, identity));
    v = op(v, lanes_from<0x142, 0xA>(v, identity));   // row_bcast 15, 31
    v = op(v, lanes_from<0x143, 0xC>(v, identity));
    return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
__device__ __forceinline__ float wave_max(float v) {
    return wave_reduce(v, -INFINITY, [](float x, float y) { return fmaxf(x, y); });
}
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
    return wave_reduce(v, (T)0, [](T x, T y) { return x + y; });
}
// The larger of three, without the quieting of signalling NaNs that fmaxf
// brings (one operation per element).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// log2(e) / T, finite.
__device__ __forceinline__ float exponent_scale(float T) {
    return fminf(fminf(1.f / T, kMaxFloat) * kLog2e, kMaxFloat);
}

// One slice's state: m, S, A in units of ln 2, how many ids come before the
// token, and the token's logit (the same in every slice of a row).
struct Slice {
    float m, S, A;
    int before;
    float lt;
};

struct LogprobsWs {
    uint64_t* best;   // [B][slices][n_top] keys, best first, 0 past the last
    Slice* part;      // [B][slices]
};

__device__ __forceinline__ void write_row(const LogprobsArgs& a, int b, float T, float m, float S,
                                          float A, int before, float lt, float logS) {
    const bool any = m > -INFINITY, has = lt > -INFINITY;
    if (a.logprob) a.logprob[b] = has ? (lt - m) / T - logS : -INFINITY;
    if (a.rank) a.rank[b] = has ? before + 1 : 0;
    if (a.lse) a.lse[b] = any ? m / T + logS : -INFINITY;
    if (a.entropy) a.entropy[b] = any ? logS - kLn2 * (A / S) : 0.f;
}
__device__ __forceinline__ void write_best(const LogprobsArgs& a, int b, int j, uint64_t key,
                                           float T, float m, float logS) {
    const size_t o = (size_t)b * a.n_top + j;
    a.top_idx[o] = key ? key_index(key) + a.v_offset : -1;
    a.top_logprob[o] = key ? (key_score(key) - m) / T - logS : -INFINITY;
}

// The row's token as a local id, and its logit (-inf: none to look at).
template <int DT>
__device__ __forceinline__ float token_logit(const LogprobsArgs& a, const uint32_t* allow_row,
                                             const typename Elem<DT>::type* row, int n, int b,
                                             int& tok) {
    tok = -1;
    if (!a.token) return -INFINITY;
    const int64_t t = (int64_t)a.token[b] - a.v_offset;
    if (a.token[b] < 0 || t < 0 || t >= n) return -INFINITY;
    tok = (int)t;
    return allowed(allow_row, tok) ? clean((float)row[tok]) : -INFINITY;
}

// The largest float below x (x finite).
__device__ __forceinline__ float below(float x) {
    return x == 0.f ? __uint_as_float(0x80000001u) : ordered_to_float(float_to_ordered(x) - 1);
}

// The n-th largest of the wave's 64 K keys (K a lane), or a smaller value that
// exactly n keys reach; reach: how many do.
template <int K>
__device__ __forceinline__ uint32_t nth_largest(const uint32_t (&k)[K], int n, int& reach) {
    uint32_t prefix = 0;
    reach = 64 * K;
    for (int bit = 31; bit >= 0 && reach != n; --bit) {
        const uint32_t cand = prefix | (1u << bit);
        int c = 0;
#pragma unroll
        for (int i = 0; i < K; ++i) c += __popcll(__ballot(k[i] >= cand));
        if (c >= n) {
            prefix = cand;
            reach = c;
        }
    }
    return prefix;
}
// The smallest id (or larger) that at least n of the 256 ids reach from below.
__device__ __forceinline__ int nth_lowest(const int* ids, int n) {
    const int lane = threadIdx.x & 63;
    uint32_t limit = 0;
    for (int bit = 30; bit >= 0; --bit) {
        const uint32_t cand = limit | ((1u << bit) - 1);
        int c = 0;
#pragma unroll
        for (int i = 0; i < kLpThreads / 64; ++i)
            c += __popcll(__ballot((uint32_t)ids[lane + 64 * i] <= cand));
        if (c < n) limit |= 1u << bit;
    }
    return (int)limit;
}

// Best alternatives of a slice held in registers.  A value that at least n
// threads' maxima reach bounds the n-th largest element from below, and only
// threads that reach it hold elements of the answer.  Each wave offers the
// ceil(n / 4)-th largest of its lanes' maxima, and the lowest of the four
// offers is such a value: the threads that reach it (somewhat over n) leave
// their elements in LDS, the elements that reach it are collected, ranked by
// counting and written best first.  Where more than kHeld threads reach it
// (values in the order of the ids, many equal values), it is raised to the
// exact n-th largest maximum, and of the threads that tie with that only those
// count whose first equal id is lowest: n threads in all.  (An element of the
// answer in another tied thread would have the n - above first ids of those
// and the above larger maxima before it.)
constexpr int kHeld = 96;    // at least kMaxAlternatives
constexpr int kKeys = 512;   // collected elements that are compacted
template <int E>
struct TopShared {
    float value[kHeld][E];
    uint64_t key[kKeys];
    int owner[kHeld];
    float tmax[kLpThreads];
    int first[kLpThreads];
    uint32_t offer[kLpWaves], alone[kLpWaves];
    int threads, count, tied, id_limit;
    uint32_t bound;
};

// This wave's offer, before the barrier that ends the maxima.  Where the row
// ends inside the slice (ragged: the same for all threads), waves without
// elements make the lowest offer worthless; the n-th largest of one wave's
// maxima is such a value too.
template <int E>
__device__ __forceinline__ void offer_bound(TopShared<E>& s, float tmax, int n, bool ragged) {
    const uint32_t k[1] = {float_to_ordered(tmax + 0.f)};
    int reach;
    const uint32_t b = nth_largest(k, (n + kLpWaves - 1) / kLpWaves, reach);
    const uint32_t alone = ragged ? nth_largest(k, n, reach) : 0;
    if ((threadIdx.x & 63) == 0) {
        s.offer[threadIdx.x >> 6] = b;
        s.alone[threadIdx.x >> 6] = alone;
    }
    if (threadIdx.x == 0) s.threads = s.count = 0;
}

// A passing thread's elements to LDS.
template <int E>
__device__ __forceinline__ void hold(TopShared<E>& s, const float (&x)[E], bool pass) {
    const int lane = threadIdx.x & 63;
    const uint64_t who = __ballot(pass);
    int slot = 0;
    if (lane == 0 && who) slot = atomicAdd(&s.threads, __popcll(who));
    slot = __builtin_amdgcn_readfirstlane(slot) + __popcll(who & ((1ull << lane) - 1));
    if (pass && slot < kHeld) {
        s.owner[slot] = threadIdx.x;
#pragma unroll
        for (int e = 0; e < E; ++e) s.value[slot][e] = x[e];
    }
}

// After that barrier; the next barrier ends it.
template <int E>
__device__ __forceinline__ uint32_t hold_offers(TopShared<E>& s, const float (&x)[E], float tmax) {
    uint32_t bound = s.offer[0];
#pragma unroll
    for (int w = 1; w < kLpWaves; ++w) bound = min(bound, s.offer[w]);
#pragma unroll
    for (int w = 0; w < kLpWaves; ++w) bound = max(bound, s.alone[w]);
    bound = max(bound, float_to_ordered(-INFINITY) + 1);   // unmasked values only
    hold(s, x, float_to_ordered(tmax + 0.f) >= bound);
    return bound;
}

// The exact bound, where the offers hold too many threads.
template <int E, typename I>
__device__ __forceinline__ uint32_t hold_exact(TopShared<E>& s, const float (&x)[E],
                                                         float tmax, I id_of, int n) {
    const int t = threadIdx.x, lane = t & 63;
    const uint32_t mine = float_to_ordered(tmax + 0.f);
    s.tmax[t] = tmax + 0.f;
    __syncthreads();
    uint32_t k[4];
    if (t < 64) {
        int reach = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) k[i] = float_to_ordered(s.tmax[lane + 64 * i]);
        const uint32_t exact = nth_largest(k, n, reach);
        const uint32_t least = float_to_ordered(-INFINITY) + 1;
        if (t == 0) {
            s.threads = 0;
            s.bound = max(exact, least);
            s.tied = reach > n && exact >= least;
            s.id_limit = 0x7FFFFFFF;
        }
    }
    __syncthreads();
    const uint32_t bound = s.bound;
    const float lo = ordered_to_float(bound);
    int first = 0x7FFFFFFF;
    if (s.tied) {   // (the same for all threads)
        int me = t;
        asm volatile("" : "+v"(me));   // the ids are formed here only
        if (mine == bound)
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (clean(x[e]) == lo) first = min(first, id_of(me, e));
        s.first[t] = first;
        __syncthreads();
        if (t < 64) {
            int above = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) above += __popcll(__ballot(k[i] > bound));
            const int limit = nth_lowest(s.first, n - above);
            if (t == 0) s.id_limit = limit;
        }
        __syncthreads();
    }
    hold(s, x, mine > bound || (mine == bound && (!s.tied || first <= s.id_limit)));
    __syncthreads();
    return bound;
}

// The held elements that reach the bound, ranked.
template <int E, typename I, typename F>
__device__ __forceinline__ void write_best_of(TopShared<E>& s, uint32_t bound, I id_of, int n,
                                              F write) {
    const int t = threadIdx.x;
    const float lo = ordered_to_float(bound);
    const int held = s.threads * E;
    auto key_of = [&](int i) {   // 0: below the bound
        const float v = s.value[i / E][i % E];
        return v >= lo ? pack_key(fminf(v, kMaxFloat) + 0.f, id_of(s.owner[i / E], i % E))
                       : (uint64_t)0;
    };
    for (int i = t; i < held; i += kLpThreads) {
        const uint64_t key = key_of(i);
        if (key) {
            const int at = atomicAdd(&s.count, 1);
            if (at < kKeys) s.key[at] = key;
        }
    }
    __syncthreads();
    const int c = s.count;
    if (c <= kKeys) {
        for (int i = t; i < c; i += kLpThreads) {
            const uint64_t key = s.key[i];
            int r = 0;
#pragma unroll 8
            for (int j = 0; j < c; ++j) r += s.key[j] > key;
            if (r < n) write(r, key);
        }
    } else {   // (many of the best in few threads)
        for (int i = t; i < held; i += kLpThreads) {
            const uint64_t key = key_of(i);
            if (!key) continue;
            int r = 0;
            for (int j = 0; j < held && r < n; ++j) r += key_of(j) > key;
            if (r < n) write(r, key);
        }
    }
    for (int i = c + t; i < n; i += kLpThreads) write(i, (uint64_t)0);
}

// One slice of kLpThreads E elements of a row.
template <int DT, int E, bool MASKED, bool TOP, bool STREAM>
__global__ __launch_bounds__(kLpThreads, 7) void logprobs_kernel(LogprobsArgs a, LogprobsWs ws,
                                                                 int slices) {
    typedef typename Elem<DT>::type T_;
    constexpr int N = Vec<DT>::kN;
    __shared__ float smax[kLpWaves], sS[kLpWaves], sA[kLpWaves];
    __shared__ int sbefore[kLpWaves];
    __shared__ std::conditional_t<TOP, TopShared<E>, char> top;
    const int n = valid_ids(a.V, a.n_valid, a.v_offset);
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int base = blockIdx.x * (kLpThreads * E);
    for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
        // (formed per row: hoisted, the ids and their tests against n would
        // take over a hundred registers)
        int lane_id = lane;
        asm volatile("" : "+v"(lane_id));
        auto chunk = [&](int j) {
            return Chunk<DT>(base + (j * kLpWaves + wave) * 64 * N, n, lane_id);
        };
        const T_* row = static_cast<const T_*>(a.logits) + (size_t)b * a.ld;
        const uint32_t* allow_row = a.allow ? a.allow + (size_t)b * ((a.V + 31) >> 5) : nullptr;
        const float T = row_temp(a.temp, b, a.flags);
        int tok;
        const float lt = token_logit<DT>(a, allow_row, row, n, b, tok);
        Vec<DT> raw[E / N];
        uint32_t bits[E / N];
#pragma unroll
        for (int j = 0; j < E / N; ++j)
            load_chunk<DT, MASKED, STREAM>(chunk(j), row, allow_row, n, raw[j], bits[j]);
        // NaN and +inf stay in x: every use below takes a NaN as masked (a
        // maximum, a comparison and a median drop it) and +inf as kMaxFloat
        float x[E];
        float tmax = -INFINITY;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[e] = raw[e / N].at(e % N);
            if constexpr (MASKED) x[e] = (bits[e / N] >> (e % N)) & 1u ? x[e] : -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < E; e += 2) tmax = max3(tmax, x[e], x[e + 1]);
        if (__any(tmax != tmax)) {   // (a signalling NaN: the maximum takes it over)
            tmax = -INFINITY;
#pragma unroll
            for (int e = 0; e < E; ++e) tmax = fmaxf(tmax, clean(x[e]));
        }
        tmax = fminf(tmax, kMaxFloat);
        const float wmax = wave_max(tmax);
        if (lane == 0) smax[wave] = wmax;
        if constexpr (TOP) offer_bound<E>(top, tmax, a.n_top, base + kLpThreads * E > n);
        __syncthreads();
        const float m = fmaxf(fmaxf(smax[0], smax[1]), fmaxf(smax[2], smax[3]));
        uint32_t bound = 0;
        if constexpr (TOP) bound = hold_offers<E>(top, x, tmax);

        const float c = exponent_scale(T);
        const float from = m > -INFINITY ? m : 0.f;
        const bool has = lt > -INFINITY;
        const float lt_below = has ? below(lt) : INFINITY;
        const float lt_over = has && lt < kMaxFloat ? lt : INFINITY;
        // (a wave whose largest is below the token has none before it)
        const bool count = a.rank && has && wmax >= lt;
        float S = 0.f, A = 0.f;
#pragma unroll
        for (int j = 0; j < E / N; ++j) {
            float S1 = 0.f, A1 = 0.f;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float d = __builtin_amdgcn_fmed3f((x[j * N + e] - from) * c, kFloor, 0.f);
                const float p = __builtin_amdgcn_exp2f(d);
                S1 += p;
                A1 = fmaf(d, p, A1);
            }
            S += S1;
            A += A1;
        }
        // ids before the token: in chunks wholly before it, those that reach
        // its logit; in chunks wholly behind it, those above
        int before = 0, mixed = 0;   // of the wave, of the lane
        if (count)
#pragma unroll
            for (int j = 0; j < E / N; ++j) {
                const Chunk<DT> ch = chunk(j);
                if (ch.whole && (tok < ch.first || tok >= ch.first + 64 * N)) {
                    const float over = tok < ch.first ? lt_over : lt_below;
#pragma unroll
                    for (int e = 0; e < N; ++e) before += __popcll(__ballot(x[j * N + e] > over));
                } else {
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        const float v = clean(x[j * N + e]);
                        mixed += v > lt || (v == lt && ch.id(e) < tok) ? 1 : 0;
                    }
                }
            }
        S = wave_sum(S);
        A = wave_sum(A);
        before += wave_sum(mixed);
        if (lane == 0) {
            sS[wave] = S;
            sA[wave] = A;
            sbefore[wave] = before;
        }
        __syncthreads();
        S = (sS[0] + sS[1]) + (sS[2] + sS[3]);
        A = (sA[0] + sA[1]) + (sA[2] + sA[3]);
        before = sbefore[0] + sbefore[1] + sbefore[2] + sbefore[3];
        const float logS = logf(S);
        if (t == 0) {
            if (slices == 1)
                write_row(a, b, T, m, S, A, before, lt, logS);
            else
                ws.part[(size_t)b * slices + blockIdx.x] = Slice{m, S, A, before, lt};
        }
        if constexpr (TOP) {
            uint64_t* out = ws.best + ((size_t)b * slices + blockIdx.x) * a.n_top;
            auto id_of = [&](int thread, int e) {
                return Chunk<DT>(base + (e / N * kLpWaves + (thread >> 6)) * 64 * N, n, thread & 63)
                    .id(e % N);
            };
            if (top.threads > kHeld) {   // (the same for all threads)
                __syncthreads();
                bound = hold_exact<E>(top, x, tmax, id_of, a.n_top);
            }
            write_best_of<E>(top, bound, id_of, a.n_top, [&](int j, uint64_t key) {
                if (slices == 1)
                    write_best(a, b, j, key, T, m, logS);
                else
                    out[j] = key;
            });
        }
        __syncthreads();   // before the next row's shared values
    }
}

// Joins the slices of a row.  Alternatives: with more than n slices the n-th
// best of their first entries bounds the row's n-th best from below, and at
// most n lists reach it; with fewer, the n-th largest of the threads' largest
// entries bounds it.  Bound by latency: everything a row needs is loaded
// before the first use (rows of more than kJoinEntries entries read theirs
// later).
template <bool STAGED>
__global__ __launch_bounds__(kLpThreads) void logprobs_join_kernel(LogprobsArgs a, LogprobsWs ws,
                                                                   int slices) {
    extern __shared__ __align__(16) uint64_t keys[];   // n_top min(n_top, slices), entries
    constexpr int kPer = kJoinEntries / kLpThreads;
    __shared__ float smax[kLpWaves], sS[kLpWaves], sA[kLpWaves];
    __shared__ int sbefore[kLpWaves];
    __shared__ int count;
    __shared__ unsigned long long bound;
    __shared__ uint32_t tbest[kLpThreads];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int n = a.n_top;
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const Slice* part = ws.part + (size_t)b * slices;
        const uint64_t* best = ws.best + (size_t)b * slices * n;
        uint64_t* entries = keys + n * min(n, slices);
        uint64_t mine[kPer];
        if constexpr (STAGED) {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (t + i * kLpThreads < slices * n) mine[i] = best[t + i * kLpThreads];
        }
        const float T = row_temp(a.temp, b, a.flags);
        Slice p{-INFINITY, 0.f, 0.f, 0, 0.f};
        if (t < slices) p = part[t];
        const float lt = part[0].lt;
        if constexpr (STAGED) {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (t + i * kLpThreads < slices * n) entries[t + i * kLpThreads] = mine[i];
        }
        if (n > 0 && slices <= n) {
            uint32_t most = 0;
            if constexpr (STAGED) {
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (t + i * kLpThreads < slices * n) most = max(most, (uint32_t)(mine[i] >> 32));
            } else {
                for (int64_t i = t; i < (int64_t)slices * n; i += kLpThreads)
                    most = max(most, (uint32_t)(best[i] >> 32));
            }
            tbest[t] = most;
        }
        float m = p.m;
        for (int i = t + kLpThreads; i < slices; i += kLpThreads) m = fmaxf(m, part[i].m);
        m = wave_max(m);
        if (lane == 0) smax[wave] = m;
        if (t == 0) {
            count = 0;
            bound = 1;
        }
        __syncthreads();
        m = fmaxf(fmaxf(smax[0], smax[1]), fmaxf(smax[2], smax[3]));
        const float c = exponent_scale(T);
        const float from = m > -INFINITY ? m : 0.f;
        float S = 0.f, A = 0.f;
        int before = 0;
        for (int i = t; i < slices; i += kLpThreads) {
            if (i != t) p = part[i];
            const float d = fmaxf((p.m - from) * c, kFloor);
            const float w = __builtin_amdgcn_exp2f(d);
            S = fmaf(p.S, w, S);
            A = fmaf(w, fmaf(d, p.S, p.A), A);
            before += p.before;
        }
        S = wave_sum(S);
        A = wave_sum(A);
        before = wave_sum(before);
        if (lane == 0) {
            sS[wave] = S;
            sA[wave] = A;
            sbefore[wave] = before;
        }
        const uint64_t* list = STAGED ? entries : best;
        if (n > 0 && slices > n)
            for (int i = t; i < slices; i += kLpThreads) {
                const uint64_t head = list[(size_t)i * n];
                int r = 0;
#pragma unroll 8
                for (int j = 0; j < slices; ++j) r += list[(size_t)j * n] > head;
                if (r == n - 1 && head) bound = head;   // (keys differ: one thread)
            }
        if (n > 0 && slices <= n && t < 64) {
            uint32_t k[4];
            int reach;
#pragma unroll
            for (int i = 0; i < 4; ++i) k[i] = tbest[lane + 64 * i];
            const uint32_t v = nth_largest(k, n, reach);
            if (t == 0 && v) bound = (unsigned long long)v << 32;
        }
        __syncthreads();
        S = (sS[0] + sS[1]) + (sS[2] + sS[3]);
        A = (sA[0] + sA[1]) + (sA[2] + sA[3]);
        before = sbefore[0] + sbefore[1] + sbefore[2] + sbefore[3];
        const float logS = logf(S);
        if (t == 0) write_row(a, b, T, m, S, A, before, lt, logS);
        if (n > 0) {
            const uint64_t lo = bound;
            for (int64_t i = t; i < (int64_t)slices * n; i += kLpThreads) {
                const uint64_t k = list[i];
                if (k >= lo) keys[atomicAdd(&count, 1)] = k;
            }
            __syncthreads();
            for (int i = t; i < count; i += kLpThreads) {
                const uint64_t key = keys[i];
                int r = 0;
#pragma unroll 8
                for (int j = 0; j < count; ++j) r += keys[j] > key;
                if (r < n) write_best(a, b, r, key, T, m, logS);
            }
            for (int i = count + t; i < n; i += kLpThreads) write_best(a, b, i, 0, T, m, logS);
        }
        __syncthreads();
    }
}

// Gradient: dl_i = 1/T [ p_i (c - g_H (ln p_i + H)) + [i = token] g_lp +
// sum_j [i = top_j] g_top_j ],  c = g_lse - g_lp - sum_j g_top_j, ln p_i = x_i
// - lse.  Bound by one read and one write of [B, V]: 2048 x 151936 bf16 in 243
// us, 5.1 TB/s.
constexpr int kGradElems = 16;   // per thread
constexpr int kSpecials = kMaxAlternatives + 1;

template <int DT, bool MASKED, bool STREAM>
__global__ __launch_bounds__(kLpThreads) void logprobs_grad_kernel(LogprobsGradArgs a) {
    typedef typename Elem<DT>::type T_;
    constexpr int N = Vec<DT>::kN;
    constexpr int kSlice = kLpThreads * kGradElems;
    __shared__ int special[kSpecials];
    __shared__ float add[kSpecials];
    __shared__ int nspecial;
    __shared__ float sum_top;
    const int n = valid_ids(a.V, a.n_valid, a.v_offset);
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int base = blockIdx.x * kSlice;
    for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
        int lane_id = lane;   // (formed per row, as above)
        asm volatile("" : "+v"(lane_id));
        // chunks of the whole row of V: masked ids are written too
        auto chunk = [&](int j) {
            return Chunk<DT>(base + (j * kLpWaves + wave) * 64 * N, a.V, lane_id);
        };
        const T_* row = static_cast<const T_*>(a.logits) + (size_t)b * a.ld;
        T_* out = static_cast<T_*>(a.grad) + (size_t)b * a.ld_grad;
        const uint32_t* allow_row = a.allow ? a.allow + (size_t)b * ((a.V + 31) >> 5) : nullptr;
        Vec<DT> raw[kGradElems / N];
        uint32_t bits[kGradElems / N];
#pragma unroll
        for (int j = 0; j < kGradElems / N; ++j)
            load_chunk<DT, MASKED, STREAM>(chunk(j), row, allow_row, a.V, raw[j], bits[j]);
        const float T = row_temp(a.temp, b, a.flags), inv_t = 1.f / T;
        float lse = a.lse[b];
        const bool ok = fabsf(lse) < INFINITY;
        lse = ok ? lse : INFINITY;   // p = 0 everywhere
        const int tok = a.g_logprob ? a.token[b] : -1;
        const float glp = tok >= 0 ? a.g_logprob[b] : 0.f;
        const float gH = a.g_entropy ? a.g_entropy[b] : 0.f;
        const float H = a.g_entropy ? a.entropy[b] : 0.f;
        // the ids of this slice that get something added, by the first wave
        if (t < 64) {
            float g = 0.f;
            int id = -1;
            if (a.g_top && t < a.n_top) {
                id = a.top_idx[(size_t)b * a.n_top + t];
                g = id >= 0 ? a.g_top[(size_t)b * a.n_top + t] : 0.f;
            }
            const float s = wave_sum(g);
            const int64_t at = (int64_t)id - a.v_offset - base;
            const bool here = ok && id >= 0 && at >= 0 && at < kSlice;
            const uint64_t who = __ballot(here);
            if (here) {
                const int slot = __popcll(who & ((1ull << t) - 1));
                special[slot] = (int)at;
                add[slot] = g * inv_t;
            }
            if (t == 0) {
                int k = __popcll(who);
                const int64_t tat = (int64_t)tok - a.v_offset - base;
                if (ok && tok >= 0 && tat >= 0 && tat < kSlice) {
                    special[k] = (int)tat;
                    add[k++] = glp * inv_t;
                }
                nspecial = k;
                sum_top = s;
            }
        }
        __syncthreads();
        const float gHt = gH * inv_t;
        const float c = ((a.g_lse ? a.g_lse[b] : 0.f) - glp - sum_top) * inv_t - gHt * H;
        const int ns = nspecial;
#pragma unroll
        for (int j = 0; j < kGradElems / N; ++j) {
            const Chunk<DT> ch = chunk(j);
            float g[N];
            bool on[N];
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float l = clean(raw[j].at(e));
                on[e] = l > -INFINITY && ch.id(e) < n;
                if constexpr (MASKED) on[e] = on[e] && ((bits[j] >> e) & 1u);
                // l / T to FP32 accuracy, and not below what e^x makes 0
                const float x0 = l * inv_t;
                const float x = fmaf(fmaf(-x0, T, l), inv_t, x0);
                const float lp = fmaxf(x - lse, -1e6f);
                g[e] = on[e] ? __builtin_amdgcn_exp2f(lp * kLog2e) * (c - gHt * lp) : 0.f;
            }
            for (int k = 0; k < ns; ++k) {
                const int at = base + special[k];
#pragma unroll
                for (int e = 0; e < N; ++e)
                    if (ch.id(e) == at && on[e]) g[e] += add[k];
            }
            if (ch.whole) {
                T_ v[N];
#pragma unroll
                for (int e = 0; e < N; ++e) v[e] = (T_)g[e];
                typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));
                u32x4 w;
                __builtin_memcpy(&w, v, 16);
                __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(out + ch.id(0)));
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e)
                    if (ch.id(e) < a.V) out[ch.id(e)] = (T_)g[e];
            }
        }
        __syncthreads();   // before the next row's special ids
    }
}

// Logits that the last-level cache cannot hold anyway are read past the caches
// (2048 x 128256 bf16: 142 against 151 us; 4096 x 32000 FP32: 89 against 97 us).
// Smaller ones may have been written just before and be there still
// (32 x 151936 FP32 again and again: 11.0 against 10.0 us).
bool past_caches(int B, int V, int dtype) {
    return (int64_t)B * V * (dtype == FS_F32 ? 4 : 2) > (int64_t)256 << 20;
}

int slice_elems(int B, int V, int cus) {
    // one slice where a workgroup holds the whole row (no second kernel); long
    // slices once they fill the chip, twice over: fewer candidates to join
    // (V = 151936 FP32, long against short: 32 rows 10.5 and 10.1 us, with 5
    // alternatives 15.4 and 19.6 us; 8 rows 8.8 and 7.3 us, 13.3 and 14.2 us)
    const int64_t one = (int64_t)kLpThreads * kLpLong;
    if (V <= kLpThreads * kLpShort) return kLpThreads * kLpShort;
    if (V <= one || (int64_t)B * ((V + one - 1) / one) >= 2 * cus) return (int)one;
    return kLpThreads * kLpShort;
}

LogprobsWs carve(const LogprobsArgs& a, void* ws, int slices) {
    LogprobsWs w;
    w.best = static_cast<uint64_t*>(ws);
    w.part = reinterpret_cast<Slice*>(w.best + (size_t)a.B * slices * a.n_top);
    return w;
}

template <int DT, int E, bool MASKED, bool STREAM>
void launch_slices(const LogprobsArgs& a, const LogprobsWs& w, int slices, hipStream_t stream) {
    const dim3 grid(slices, a.B < kMaxGridY ? a.B : kMaxGridY);
    if (a.n_top > 0)
        hipLaunchKernelGGL((logprobs_kernel<DT, E, MASKED, true, STREAM>), grid, dim3(kLpThreads), 0,
                           stream, a, w, slices);
    else
        hipLaunchKernelGGL((logprobs_kernel<DT, E, MASKED, false, STREAM>), grid, dim3(kLpThreads), 0,
                           stream, a, w, slices);
}

template <int DT>
void launch_type(const LogprobsArgs& a, const LogprobsWs& w, int slices, bool lng,
                 hipStream_t stream) {
    if (lng && past_caches(a.B, a.V, a.dtype))
        a.allow ? launch_slices<DT, kLpLong, true, true>(a, w, slices, stream)
                : launch_slices<DT, kLpLong, false, true>(a, w, slices, stream);
    else if (lng)
        a.allow ? launch_slices<DT, kLpLong, true, false>(a, w, slices, stream)
                : launch_slices<DT, kLpLong, false, false>(a, w, slices, stream);
    else
        a.allow ? launch_slices<DT, kLpShort, true, false>(a, w, slices, stream)
                : launch_slices<DT, kLpShort, false, false>(a, w, slices, stream);
}

}  // namespace

size_t logprobs_ws_bytes(int B, int V, int n_top, int cus) {
    const int per = slice_elems(B, V, cus);
    const size_t slices = V > 0 ? ((size_t)V + per - 1) / per : 1;
    return slices > 1 ? (size_t)B * slices * (sizeof(Slice) + 8 * (size_t)n_top) : 0;
}

hipError_t launch_logprobs(const LogprobsArgs& a, void* ws, int cus, hipStream_t stream) {
    const int per = slice_elems(a.B, a.V, cus);
    const int slices = a.V > 0 ? (int)(((int64_t)a.V + per - 1) / per) : 1;
    const LogprobsWs w = carve(a, ws, slices);
    const bool lng = per == kLpThreads * kLpLong;
    if (a.dtype == FS_F32)
        launch_type<FS_F32>(a, w, slices, lng, stream);
    else if (a.dtype == FS_BF16)
        launch_type<FS_BF16>(a, w, slices, lng, stream);
    else
        launch_type<FS_F16>(a, w, slices, lng, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || slices == 1) return e;
    // at most 32 KiB of candidates and 16 KiB of entries
    const int64_t entries = (int64_t)slices * a.n_top;
    const bool staged = entries <= kJoinEntries;
    const size_t lds = 8 * ((size_t)a.n_top * std::min(a.n_top, slices) + (staged ? entries : 0));
    if (staged)
        hipLaunchKernelGGL(logprobs_join_kernel<true>, dim3(a.B), dim3(kLpThreads), lds, stream, a,
                           w, slices);
    else
        hipLaunchKernelGGL(logprobs_join_kernel<false>, dim3(a.B), dim3(kLpThreads), lds, stream, a,
                           w, slices);
    return hipGetLastError();
}

hipError_t launch_logprobs_grad(const LogprobsGradArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)(((int64_t)a.V + kLpThreads * kGradElems - 1) / (kLpThreads * kGradElems)),
                    a.B < kMaxGridY ? a.B : kMaxGridY);
    const bool past = past_caches(a.B, a.V, a.dtype);
#define FS_LG(DT_, M_, S_)                                                                       \
    if (a.dtype == DT_ && (a.allow != nullptr) == M_ && past == S_)                              \
        hipLaunchKernelGGL((logprobs_grad_kernel<DT_, M_, S_>), grid, dim3(kLpThreads), 0, stream, a);
#define FS_LG_TYPE(DT_) \
    FS_LG(DT_, false, false) FS_LG(DT_, false, true) FS_LG(DT_, true, false) FS_LG(DT_, true, true)
    FS_LG_TYPE(FS_F32)
    FS_LG_TYPE(FS_BF16)
    FS_LG_TYPE(FS_F16)
#undef FS_LG_TYPE
#undef FS_LG
    return hipGetLastError();
}

}  // namespace fs
