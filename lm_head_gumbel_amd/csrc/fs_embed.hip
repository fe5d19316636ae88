// Embedding of token ids, out[n] = scale W[ids[n]], and its gradient,
// dW[v] = scale sum of g[n] over the n with ids[n] = v.
//
// Both are bound by memory: a read and a write of [N, d], and for the gradient
// one read of g and one write of dW.  The gradient sorts the tokens by id
// (stable radix sort, so equal ids keep the order of n), cuts the sorted list
// into chunks, sums each chunk's runs of equal ids in FP32 and
// writes the runs that lie inside a chunk straight to dW; runs that cross a
// chunk's end leave partial rows, which a last kernel adds up in order.  The
// order of every sum follows from the ids alone.
//
// MI355X: 16384 tokens of 5120 bf16 in 44 us captured (5.4 TB/s; 56 us with
// inputs that no cache holds); the gradient of 16384 tokens of 4096 bf16 to an
// FP32 dW of 151936 rows in 569 us, 4.6 TB/s.
#include <algorithm>

#include "fs_vocab.h"

namespace fs {

namespace {

constexpr int kEmThreads = 256;

// Elements of 16 bytes of a type, from any element-aligned address.
template <int DT>
struct Row16 {
    typedef typename Elem<DT>::type E;
    static constexpr int kN = 16 / (int)sizeof(E);
};
// Elements k .. k + kN - 1 of a row of d in FP32 (0 past the end).
template <int DT>
__device__ __forceinline__ void load_row(const typename Elem<DT>::type* row, int k, int d,
                                         float* x) {
    constexpr int N = Row16<DT>::kN;
    typename Elem<DT>::type v[N];
    if (k + N <= d) {
        __builtin_memcpy(v, row + k, 16);
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = (float)v[e];
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = k + e < d ? (float)row[k + e] : 0.f;
    }
}
// N values to elements k .. of a row of d; STREAM: past the caches, for what
// is not read again soon.
template <int DT, int N, bool STREAM = false>
__device__ __forceinline__ void store_row(typename Elem<DT>::type* row, int k, int d,
                                          const float* x) {
    typename Elem<DT>::type v[N];
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = (typename Elem<DT>::type)x[e];
    if (k + N <= d) {
        if constexpr (STREAM && sizeof(v) == 16) {
            typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));
            u32x4 w;
            __builtin_memcpy(&w, v, 16);
            __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(row + k));
        } else {
            __builtin_memcpy(row + k, v, sizeof(v));
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (k + e < d) row[k + e] = v[e];
    }
}

// `lanes` threads (a power of two up to 256) per row, kEmThreads / lanes rows
// per workgroup.
template <int DT>
__global__ __launch_bounds__(kEmThreads) void embed_kernel(EmbedArgs a, int lanes) {
    typedef typename Elem<DT>::type E;
    constexpr int N = Row16<DT>::kN;
    const int per = kEmThreads / lanes;
    const int sub = threadIdx.x / lanes, lane = threadIdx.x % lanes;
    for (int64_t n = (int64_t)blockIdx.x * per + sub; n < a.N; n += (int64_t)gridDim.x * per) {
        const int64_t j = (int64_t)a.ids[n] - a.v_offset;
        const bool in = j >= 0 && j < a.V;
        const E* row = static_cast<const E*>(a.W) + (in ? (size_t)j * a.d : 0);
        E* out = static_cast<E*>(a.out) + (size_t)n * a.d;
        for (int k = lane * N; k < a.d; k += 2 * lanes * N) {
            float x[2][N];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int e = 0; e < N; ++e) x[u][e] = 0.f;
                const int ku = k + u * lanes * N;
                if (in && ku < a.d) load_row<DT>(row, ku, a.d, x[u]);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int ku = k + u * lanes * N;
                // (a row outside the shard is 0, also with an infinite scale)
#pragma unroll
                for (int e = 0; e < N; ++e) x[u][e] = in ? a.scale * x[u][e] : 0.f;
                if (ku < a.d) store_row<DT, N, true>(out, ku, a.d, x[u]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// stable radix sort of (id, n): digits of kDigitBits, tiles of kTile tokens
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kRounds = 4;                        // tokens per thread
constexpr int kTile = kSortThreads * kRounds;     // 4096
constexpr int kDigitBits = 9;
constexpr int kDigits = 1 << kDigitBits;

// The sort key of an id: its row of this shard, or V for none.
__device__ __forceinline__ uint32_t row_key_of(int32_t id, int v_offset, int V) {
    const int64_t j = (int64_t)id - v_offset;
    return j >= 0 && j < V ? (uint32_t)j : (uint32_t)V;
}

struct SortShared {
    uint32_t wave[kSortWaves][kDigits];   // per wave: count, then offset
    uint32_t total[kDigits];
    uint32_t base[kDigits];
    uint32_t part[kSortWaves];
};

// Ranks a tile's digits (digit[r] of token (wave 64 kRounds + 64 r + lane),
// -1: no token) among the equal digits before them in the tile: rank[r] within
// the wave, s.wave[wave][digit] the tokens of the waves before, s.total the
// tile's counts.
__device__ __forceinline__ void rank_tile(SortShared& s, const int (&digit)[kRounds],
                                          uint32_t (&rank)[kRounds]) {
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    for (int i = t; i < kSortWaves * kDigits; i += kSortThreads) (&s.wave[0][0])[i] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const bool on = digit[r] >= 0;
        uint64_t same = __ballot(on);
#pragma unroll
        for (int b = 0; b < kDigitBits; ++b) {
            const uint64_t bit = __ballot((digit[r] >> b) & 1);
            same &= (digit[r] >> b) & 1 ? bit : ~bit;
        }
        const uint64_t below = same & ((1ull << lane) - 1);
        uint32_t before = 0;
        if (on) before = s.wave[wave][digit[r]];
        rank[r] = before + __popcll(below);
        // the lanes of a wave read before the first of each digit writes
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (on && below == 0) s.wave[wave][digit[r]] = before + __popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    if (t < kDigits) {
        uint32_t sum = 0;
        for (int w = 0; w < kSortWaves; ++w) {
            const uint32_t c = s.wave[w][t];
            s.wave[w][t] = sum;
            sum += c;
        }
        s.total[t] = sum;
    }
    __syncthreads();
}

// s.base = exclusive prefix sums of v over the digits (thread t < kDigits: v).
__device__ __forceinline__ void scan_digits(SortShared& s, uint32_t v) {
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    uint32_t x = t < kDigits ? v : 0;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t y = __shfl_up(x, o, 64);
        if (lane >= o) x += y;
    }
    if (lane == 63) s.part[wave] = x;
    __syncthreads();
    if (t < kDigits) {
        uint32_t before = 0;
        for (int w = 0; w < wave; ++w) before += s.part[w];
        s.base[t] = before + x - v;
    }
    __syncthreads();
}

// Few tokens: each finds its place by counting the keys before it, four
// threads a token (a quarter of the keys each).
constexpr int kFew = 1024;
constexpr int kFewPer = kEmThreads / 4;   // tokens per workgroup
__global__ __launch_bounds__(kEmThreads) void sort_few_kernel(const int32_t* ids, int N,
                                                              int v_offset, int V,
                                                              uint32_t* out_key,
                                                              uint32_t* out_pos) {
    __shared__ __align__(16) uint32_t key[kFew];
#pragma unroll
    for (int i = 0; i < kFew / kEmThreads; ++i) {
        const int j = i * kEmThreads + threadIdx.x;
        key[j] = j < N ? row_key_of(ids[j], v_offset, V) : ~0u;
    }
    __syncthreads();
    const int n = min((int)(blockIdx.x * kFewPer + threadIdx.x / 4), N - 1);
    const int part = threadIdx.x % 4;
    const uint32_t mine = key[n];
    int at = 0;
#pragma unroll 4
    for (int i = part * 4; i < N; i += 16) {
        const uint4 k = *reinterpret_cast<const uint4*>(key + i);
        at += (k.x < mine || (k.x == mine && i < n)) + (k.y < mine || (k.y == mine && i + 1 < n)) +
              (k.z < mine || (k.z == mine && i + 2 < n)) + (k.w < mine || (k.w == mine && i + 3 < n));
    }
    at += __shfl_xor(at, 1, 64);
    at += __shfl_xor(at, 2, 64);
    if (part == 0 && blockIdx.x * kFewPer + threadIdx.x / 4 < N) {
        out_key[at] = mine;
        out_pos[at] = n;
    }
}

// One tile: the whole sort in LDS.
__global__ __launch_bounds__(kSortThreads) void sort_small_kernel(const int32_t* ids, int N,
                                                                  int v_offset, int V, int passes,
                                                                  uint32_t* out_key,
                                                                  uint32_t* out_pos) {
    __shared__ SortShared s;
    __shared__ uint32_t key[kTile], pos[kTile];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int first = wave * 64 * kRounds + lane;
    uint32_t k[kRounds], p[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int n = first + 64 * r;
        k[r] = n < N ? row_key_of(ids[n], v_offset, V) : 0;
        p[r] = n;
    }
    for (int pass = 0; pass < passes; ++pass) {
        int digit[kRounds];
        uint32_t rank[kRounds];
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
            digit[r] = first + 64 * r < N ? (int)((k[r] >> (pass * kDigitBits)) & (kDigits - 1)) : -1;
        rank_tile(s, digit, rank);
        scan_digits(s, t < kDigits ? s.total[t] : 0);
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
            if (digit[r] >= 0) {
                const uint32_t at = s.base[digit[r]] + s.wave[wave][digit[r]] + rank[r];
                key[at] = k[r];
                pos[at] = p[r];
            }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int n = first + 64 * r;
            if (n < N) {
                k[r] = key[n];
                p[r] = pos[n];
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int n = first + 64 * r;
        if (n < N) {
            out_key[n] = k[r];
            out_pos[n] = p[r];
        }
    }
}

// One pass over many tiles.  The tokens come from ids (first pass) or from the
// last pass's arrays.
struct SortPass {
    const int32_t* ids;
    const uint32_t* key;
    const uint32_t* pos;
    int N, v_offset, V, shift;
};
__device__ __forceinline__ uint32_t pass_key(const SortPass& a, int n) {
    return a.ids ? row_key_of(a.ids[n], a.v_offset, a.V) : a.key[n];
}

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortPass a, uint32_t* hist) {
    __shared__ uint32_t count[kDigits];
    const int t = threadIdx.x;
    if (t < kDigits) count[t] = 0;
    __syncthreads();
    for (int r = 0; r < kRounds; ++r) {
        const int n = blockIdx.x * kTile + r * kSortThreads + t;
        if (n < a.N) atomicAdd(&count[(pass_key(a, n) >> a.shift) & (kDigits - 1)], 1u);
    }
    __syncthreads();
    if (t < kDigits) hist[(size_t)blockIdx.x * kDigits + t] = count[t];
}

__global__ __launch_bounds__(kSortThreads) void sort_scatter_kernel(SortPass a,
                                                                    const uint32_t* hist,
                                                                    uint32_t* out_key,
                                                                    uint32_t* out_pos) {
    __shared__ SortShared s;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int first = blockIdx.x * kTile + wave * 64 * kRounds + lane;
    uint32_t k[kRounds], p[kRounds], rank[kRounds];
    int digit[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int n = first + 64 * r;
        k[r] = n < a.N ? pass_key(a, n) : 0;
        p[r] = n < a.N && a.pos ? a.pos[n] : (uint32_t)n;
        digit[r] = n < a.N ? (int)((k[r] >> a.shift) & (kDigits - 1)) : -1;
    }
    uint32_t all = 0, before = 0;
    if (t < kDigits)
        for (int b = 0; b < (int)gridDim.x; ++b) {
            const uint32_t c = hist[(size_t)b * kDigits + t];
            before += b < (int)blockIdx.x ? c : 0;
            all += c;
        }
    rank_tile(s, digit, rank);
    scan_digits(s, all);
    if (t < kDigits) s.base[t] += before;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
        if (digit[r] >= 0) {
            const uint32_t at = s.base[digit[r]] + s.wave[wave][digit[r]] + rank[r];
            out_key[at] = k[r];
            out_pos[at] = p[r];
        }
}

// ---------------------------------------------------------------------------
// sums of the runs of equal ids
// ---------------------------------------------------------------------------
// Sorted tokens per chunk.  A chunk's rows are read kAhead at a time, one
// latency each, so chunks are that short until they fill the chip; longer ones
// write fewer partial rows.  (bf16, short against long: 16000 tokens of 256
// 35 and 45 us, of 1024 61 and 69 us; 64000 of 1024 102 and 86 us.)
constexpr int kAhead = 8;
constexpr int kMaxChunk = 32;
int chunk_for(int N, int d) { return (int64_t)N * d <= (int64_t)1 << 24 ? kAhead : kMaxChunk; }
constexpr int kZeroRows = 64;   // rows of dW that one workgroup fills with zeros

struct SumArgs {
    const uint32_t* key;   // sorted rows (V: none), and the tokens' n
    const uint32_t* pos;
    const void* g;
    void* dW;
    float* part;           // [chunks][2][d]: head (a run from before), tail (a run going on)
    int N, d, V;
    int chunk;             // sorted tokens per chunk
    float scale;
    int accumulate;
    int lanes;             // threads per chunk and column block (a power of two)
    int col_blocks;
    int zero_lanes;        // threads per row that fills with zeros (a power of two)
    int sum_wgs;           // workgroups that sum; the others fill with zeros
};

// A finished sum to dW.
template <int DO, int N>
__device__ __forceinline__ void write_sum(const SumArgs& a, uint32_t row, int k,
                                          const float (&acc)[N]) {
    typedef typename Elem<DO>::type O;
    O* out = static_cast<O*>(a.dW) + (size_t)row * a.d;
    float x[N];
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = a.scale * acc[e];
    if (a.accumulate) {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (k + e < a.d) x[e] += (float)out[k + e];
    }
    store_row<DO, N>(out, k, a.d, x);
}

// Zeros in the rows row0 .. row0 + kZeroRows - 1 that no token names: 256
// probes of the sorted keys narrow the rows' tokens to a stretch, which is
// read and marked.
template <int DO>
__device__ void zero_rows(const SumArgs& a, uint32_t row0) {
    typedef typename Elem<DO>::type O;
    constexpr int N = 16 / (int)sizeof(O);
    __shared__ uint32_t named[kZeroRows / 32];
    const int t = threadIdx.x;
    if (t < kZeroRows / 32) named[t] = 0;
    const int step = max(1, (a.N + kEmThreads - 1) / kEmThreads);
    const bool in = (int64_t)t * step < a.N;
    const uint32_t probe = in ? a.key[t * step] : ~0u;
    const int below = __syncthreads_count(in && probe < row0);
    const int upto = __syncthreads_count(in && probe < row0 + kZeroRows);
    const int i1 = (int)min((int64_t)upto * step, (int64_t)a.N);
    for (int i = max(0, (below - 1) * step) + t; i < i1; i += kEmThreads) {
        const uint32_t r = a.key[i] - row0;
        if (r < kZeroRows) atomicOr(&named[r / 32], 1u << (r % 32));
    }
    __syncthreads();
    const float zero[N] = {};
    for (int r = t / a.zero_lanes; r < kZeroRows; r += kEmThreads / a.zero_lanes) {
        const uint32_t row = row0 + r;
        if (row >= (uint32_t)a.V || ((named[r / 32] >> (r % 32)) & 1u)) continue;
        O* out = static_cast<O*>(a.dW) + (size_t)row * a.d;
        for (int k = t % a.zero_lanes * N; k < a.d; k += a.zero_lanes * N)
            store_row<DO, N, true>(out, k, a.d, zero);
    }
    __syncthreads();   // before the next rows' marks
}
// Workgroup i of the wgs behind a kernel's own that fill with zeros.
template <int DO>
__device__ void zero_part(const SumArgs& a, int i, int wgs) {
    for (int64_t r = (int64_t)i * kZeroRows; r < a.V; r += (int64_t)wgs * kZeroRows)
        zero_rows<DO>(a, (uint32_t)r);
}

// Sums of the chunks: `lanes` threads per chunk and column block.
template <int DT, int DO>
__global__ __launch_bounds__(kEmThreads) void embed_sum_kernel(SumArgs a) {
    typedef typename Elem<DT>::type E;
    constexpr int N = Row16<DT>::kN;
    if ((int)blockIdx.x >= a.sum_wgs) {
        zero_part<DO>(a, (int)blockIdx.x - a.sum_wgs, (int)gridDim.x - a.sum_wgs);
        return;
    }
    const int per = kEmThreads / a.lanes;   // chunks per workgroup
    const int sub = threadIdx.x / a.lanes, lane = threadIdx.x % a.lanes;
    const int64_t c0 = (int64_t)(blockIdx.x / a.col_blocks) * per;
    const int k = ((int)(blockIdx.x % a.col_blocks) * a.lanes + lane) * N;
    // the chunks' rows and tokens, with the row before the first and the one
    // behind the last (none: ~0)
    extern __shared__ uint32_t list[];   // per a.chunk + 2 rows, per a.chunk tokens
    uint32_t* toks = list + per * a.chunk + 2;
    const int64_t base = c0 * a.chunk;
    for (int i = threadIdx.x; i < per * a.chunk + 2; i += kEmThreads) {
        const int64_t at = base + i - 1;
        list[i] = at >= 0 && at < a.N ? a.key[at] : ~0u;
    }
    for (int i = threadIdx.x; i < per * a.chunk; i += kEmThreads)
        toks[i] = base + i < a.N ? a.pos[base + i] : 0;
    __syncthreads();
    const int64_t c = c0 + sub;
    if (c * a.chunk >= a.N || k >= a.d) return;
    const uint32_t* rows = list + sub * a.chunk + 1;
    const uint32_t* tok = toks + sub * a.chunk;
    const int len = (int)min((int64_t)a.chunk, a.N - c * a.chunk);
    const E* g = static_cast<const E*>(a.g);
    float acc[N] = {};
    bool head = rows[-1] == rows[0];   // the first run began in an earlier chunk
    for (int i = 0; i < len; i += kAhead) {
        float x[kAhead][N];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (i + u < len && rows[i + u] < (uint32_t)a.V)
                load_row<DT>(g + (size_t)tok[i + u] * a.d, k, a.d, x[u]);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (i + u >= len || rows[i + u] >= (uint32_t)a.V) break;   // (none: sorted last)
            const uint32_t row = rows[i + u];
#pragma unroll
            for (int e = 0; e < N; ++e) acc[e] += x[u][e];
            const bool more = rows[i + u + 1] == row;   // the run goes on
            if (more && i + u + 1 < len) continue;
            if (head || more)
                store_row<FS_F32, N>(a.part + ((size_t)c * 2 + (head ? 0 : 1)) * a.d, k, a.d, acc);
            else
                write_sum<DO, N>(a, row, k, acc);
            head = false;
#pragma unroll
            for (int e = 0; e < N; ++e) acc[e] = 0.f;
        }
    }
}

// Runs over several chunks: the chunk where a run begins adds up its parts.
// (The zeros ride here, where they hide the long runs' latency.)
template <int DT, int DO>
__global__ __launch_bounds__(kEmThreads) void embed_join_kernel(SumArgs a, int chunks) {
    constexpr int N = Row16<DT>::kN;
    if ((int)blockIdx.x >= a.sum_wgs) {
        zero_part<DO>(a, (int)blockIdx.x - a.sum_wgs, (int)gridDim.x - a.sum_wgs);
        return;
    }
    const int per = kEmThreads / a.lanes;
    const int sub = threadIdx.x / a.lanes, lane = threadIdx.x % a.lanes;
    const int64_t c = (int64_t)(blockIdx.x / a.col_blocks) * per + sub;
    const int k = ((int)(blockIdx.x % a.col_blocks) * a.lanes + lane) * N;
    if (c + 1 >= chunks || k >= a.d) return;
    const int64_t next = (c + 1) * a.chunk;   // the next chunk's first token
    const uint32_t row = a.key[next];
    if (row >= (uint32_t)a.V || a.key[next - 1] != row) return;   // no run crosses
    if (c > 0 && a.key[next - a.chunk - 1] == row) return;         // it began earlier
    auto load_part = [&](int64_t chunk, int tail, float* x) {
        const float* p = a.part + ((size_t)chunk * 2 + tail) * a.d;
        load_row<FS_F32>(p, k, a.d, x);
        if constexpr (N > 4) load_row<FS_F32>(p, k + 4, a.d, x + 4);
    };
    float acc[N];
    load_part(c, 1, acc);
    bool more = true;
    for (int64_t j = c + 1; more; j += kAhead) {
        float x[kAhead][N];
        bool on[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            on[u] = j + u < chunks && a.key[(j + u) * a.chunk] == row;
            if (on[u]) load_part(j + u, 0, x[u]);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            more = more && on[u];
            if (more)
#pragma unroll
                for (int e = 0; e < N; ++e) acc[e] += x[u][e];
        }
    }
    write_sum<DO, N>(a, row, k, acc);
}

// The smallest power of two >= n, at most 256.
int lanes_for(int n) {
    int l = 1;
    while (l < n && l < kEmThreads) l *= 2;
    return l;
}

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

struct GradWs {
    size_t key[2], pos[2], hist, part, total;
};
GradWs grad_ws(int N, int d) {
    GradWs w;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t r = off;
        off += align_up(bytes);
        return r;
    };
    const size_t tiles = ((size_t)N + kTile - 1) / kTile;
    const size_t chunks = ((size_t)N + chunk_for(N, d) - 1) / chunk_for(N, d);
    for (int i = 0; i < 2; ++i) {
        w.key[i] = take((size_t)N * 4);
        w.pos[i] = take((size_t)N * 4);
    }
    w.hist = take(tiles * kDigits * 4);
    w.part = take(chunks > 1 ? chunks * 2 * d * 4 : 0);
    w.total = off;
    return w;
}

template <int DT, int DO>
hipError_t launch_sums(const EmbedGradArgs& a, SumArgs s, hipStream_t stream) {
    const int N = Row16<DT>::kN;
    const int vecs = (a.d + N - 1) / N;
    s.lanes = std::max(4, lanes_for(vecs));   // (at most 64 chunks' lists per workgroup)
    s.col_blocks = (vecs + s.lanes - 1) / s.lanes;
    s.chunk = chunk_for(a.N, a.d);
    const int chunks = (a.N + s.chunk - 1) / s.chunk;
    const int per = kEmThreads / s.lanes;
    s.sum_wgs = (chunks + per - 1) / per * s.col_blocks;
    const int zero_wgs =
        a.accumulate ? 0 : (int)std::min(((int64_t)a.V + kZeroRows - 1) / kZeroRows, kMaxGridX);
    const int zn = 16 / (int)sizeof(typename Elem<DO>::type);
    s.zero_lanes = lanes_for((a.d + zn - 1) / zn);
    const size_t lds = 4 * (size_t)(2 * per * s.chunk + 2);   // at most 16 KiB + 8
    const int here = chunks < 2 ? zero_wgs : 0;
    if (s.sum_wgs + here > 0)
        hipLaunchKernelGGL((embed_sum_kernel<DT, DO>), dim3(s.sum_wgs + here), dim3(kEmThreads),
                           lds, stream, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || chunks < 2) return e;
    hipLaunchKernelGGL((embed_join_kernel<DT, DO>), dim3(s.sum_wgs + zero_wgs), dim3(kEmThreads), 0,
                       stream, s, chunks);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_embed(const EmbedArgs& a, hipStream_t stream) {
    const int vec = 16 / (a.dtype == FS_F32 ? 4 : 2);
    const int lanes = lanes_for((a.d + vec - 1) / vec);
    const int per = kEmThreads / lanes;
    const dim3 grid((a.N + per - 1) / per);
    if (a.dtype == FS_F32)
        hipLaunchKernelGGL(embed_kernel<FS_F32>, grid, dim3(kEmThreads), 0, stream, a, lanes);
    else if (a.dtype == FS_BF16)
        hipLaunchKernelGGL(embed_kernel<FS_BF16>, grid, dim3(kEmThreads), 0, stream, a, lanes);
    else
        hipLaunchKernelGGL(embed_kernel<FS_F16>, grid, dim3(kEmThreads), 0, stream, a, lanes);
    return hipGetLastError();
}

size_t embed_grad_ws_bytes(int N, int d) { return grad_ws(N, d).total; }

hipError_t launch_embed_grad(const EmbedGradArgs& a, void* ws, hipStream_t stream) {
    const GradWs lay = grad_ws(a.N, a.d);
    char* base = static_cast<char*>(ws);
    auto u32 = [&](size_t off) { return reinterpret_cast<uint32_t*>(base + off); };
    // digits of 0 .. V
    int passes = 1;
    while (passes * kDigitBits < 32 && ((uint32_t)a.V >> (passes * kDigitBits)) != 0) ++passes;
    int at = 0;   // the arrays that hold the sorted tokens
    if (a.N > 0 && a.N <= kFew) {
        hipLaunchKernelGGL(sort_few_kernel, dim3((a.N + kFewPer - 1) / kFewPer),
                           dim3(kEmThreads), 0, stream, a.ids, a.N, a.v_offset, a.V, u32(lay.key[0]), u32(lay.pos[0]));
    } else if (a.N > 0 && a.N <= kTile) {
        hipLaunchKernelGGL(sort_small_kernel, dim3(1), dim3(kSortThreads), 0, stream, a.ids, a.N,
                           a.v_offset, a.V, passes, u32(lay.key[0]), u32(lay.pos[0]));
    } else if (a.N > 0) {
        const int tiles = (a.N + kTile - 1) / kTile;
        for (int pass = 0; pass < passes; ++pass) {
            const SortPass p{pass == 0 ? a.ids : nullptr, u32(lay.key[at ^ 1]), pass == 0 ? nullptr : u32(lay.pos[at ^ 1]),
                             a.N, a.v_offset, a.V, pass * kDigitBits};
            hipLaunchKernelGGL(sort_count_kernel, dim3(tiles), dim3(kSortThreads), 0, stream, p,
                               u32(lay.hist));
            hipLaunchKernelGGL(sort_scatter_kernel, dim3(tiles), dim3(kSortThreads), 0, stream, p,
                               u32(lay.hist), u32(lay.key[at]), u32(lay.pos[at]));
            at ^= 1;
        }
        at ^= 1;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    SumArgs s{};
    s.key = u32(lay.key[at]);
    s.pos = u32(lay.pos[at]);
    s.g = a.g;
    s.dW = a.dW;
    s.part = reinterpret_cast<float*>(base + lay.part);
    s.N = a.N;
    s.d = a.d;
    s.V = a.V;
    s.scale = a.scale;
    s.accumulate = a.accumulate;
#define FS_EG(DT_, DO_) \
    if (a.dtype == DT_ && a.dw_dtype == DO_) return launch_sums<DT_, DO_>(a, s, stream);
    FS_EG(FS_F32, FS_F32)
    FS_EG(FS_BF16, FS_F32)
    FS_EG(FS_BF16, FS_BF16)
    FS_EG(FS_F16, FS_F32)
    FS_EG(FS_F16, FS_F16)
#undef FS_EG
    return hipErrorInvalidValue;
}

}  // namespace fs
