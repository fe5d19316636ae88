// Logits of a W held in 4 bits with a scale (and a zero point) per group of
// consecutive k:
//   l[b, j] = sum over groups g of s[j, g] (sum_{k in g} H[b, k] q[j, k]
//                                           - z[j, g] sum_{k in g} H[b, k]).
//
// Bound by the read of W (d / 2 bytes a row) up to about 64 columns, so the
// kernel is built around keeping W loads in flight and few vector operations
// per weight.  Each wave owns 16-row blocks of W and all columns of its
// workgroup: lane (r, q) reads 16 bytes = 32 weights of row r, so one load
// instruction of a wave brings 128 k of 16 rows.  A 32-bit word of 8 weights
// becomes 8 bfloat16 values 16 + w without a conversion: bfloat16 has 7
// mantissa bits, so in [16, 32) the four bits of w are bits 3..6; a shift and
// one and-or make two of them.  v_mfma_f32_16x16x32_bf16 then forms
// sum H (16 + w) per group in FP32, started from -(16 + z) sum H (both sums
// in FP32: no weight is rounded), and one multiply-add with s adds the group
// to the row's total.  H lies in LDS in operand order, its k permuted as the
// words unpack.
//
// MI355X: B=1, d=4096, V=151936, group 128 in 65 us, 5.0 TB/s, what a large
// copy reaches.  B=64, d=5120, V=152057, group 64 in 221 to 243 us, 410 to 450
// TFLOP/s: bound by the vector and LDS instructions beside the matrix ones
// (unpacking, a start and a multiply-add per group and tile) with two waves a
// SIMD.
#include "fs_vocab.h"

#include "fs_internal.h"
#include "fs_mfma.h"

namespace fs {

namespace {

constexpr int kQWaves = 8;
constexpr int kQThreads = 64 * kQWaves;
constexpr int kQBlock = 128;   // k of one load instruction
constexpr int kQDepth = 4;     // loads of a row block in flight per wave

// Blocks of k whose scales a wave holds in LDS: all kQDepth, or half of them
// where several column blocks and groups of 32 leave no room for more.
__host__ __device__ constexpr int pair_slots(int nb, int ns) {
    return nb >= 2 && ns == 4 ? kQDepth / 2 : kQDepth;
}

struct QuantPlan {
    int nb;        // 16-column blocks per workgroup
    int C;         // columns stored in LDS
    int nkb;       // k blocks of 128, padded to a multiple of kQDepth ksplit
    int KC;        // k blocks per LDS chunk
    int nchunks;
    int mr;        // 16-row blocks per wave and pass: 2 where H passes through LDS
                   // in chunks, which both use; else 1 (two measured the same or
                   // up to 12% slower, with half the waves a SIMD can hold)
    int ksplit;    // waves that share a row block (resident only)
    bool chunked;  // H passes through LDS in chunks (else it stays there whole)
    int G;         // workgroups along V
    int per_pass;  // 16-row blocks per workgroup and pass
    int grid_y;
    size_t h_bytes, s_bytes;   // LDS: one chunk of H, and of its sums
    size_t pair_off, lds;      // the waves' scales, and all
};

// k of (operand step j, lane quarter q) within a block of 128, for groups of
// 32 SUB: which word of which lane reaches the step (see transpose_words).
template <int SUB>
__host__ __device__ constexpr int piece_of(int j, int q) {   // k / 8
    return SUB == 4   ? q * 4 + j
           : SUB == 1 ? j * 4 + q
                      : ((j >> 1) * 2 + (q & 1)) * 4 + (q >> 1) * 2 + (j & 1);
}

// Lane (r, q) holds words 0..3 of the 32 k at 32 q.  Groups of 128 take them
// as they are: step j has word j of every quarter.  Groups of 32 need steps
// whose four quarters lie in one group: the 4 x 4 transpose of words and
// quarters.  Groups of 64: the halves of the wave swapped, which is its first
// half.
template <int SUB>
__device__ __forceinline__ u32x4 transpose_words(u32x4 w) {
    if constexpr (SUB <= 2) {
        const auto a = __builtin_amdgcn_permlane32_swap(w.x, w.z, false, false);
        const auto b = __builtin_amdgcn_permlane32_swap(w.y, w.w, false, false);
        w = u32x4{a[0], b[0], a[1], b[1]};
    }
    if constexpr (SUB == 1) {
        const auto a = __builtin_amdgcn_permlane16_swap(w.x, w.y, false, false);
        const auto b = __builtin_amdgcn_permlane16_swap(w.z, w.w, false, false);
        w = u32x4{a[0], a[1], b[0], b[1]};
    }
    return w;
}

// 8 weights -> bfloat16 16 + w, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ bf16x8 unpack_word(uint32_t w, uint32_t mask, uint32_t sixteen) {
    return __builtin_bit_cast(
        bf16x8, u32x4{((w << 3) & mask) | sixteen, ((w >> 1) & mask) | sixteen,
                      ((w >> 5) & mask) | sixteen, ((w >> 9) & mask) | sixteen});
}

// The same order for 8 bfloat16 of H.
__device__ __forceinline__ u32x4 permute_h(u32x4 h) {
    constexpr uint32_t kLow = 0x05040100u, kHigh = 0x07060302u;   // halves of (second, first)
    return u32x4{__builtin_amdgcn_perm(h.z, h.x, kLow), __builtin_amdgcn_perm(h.z, h.x, kHigh),
                 __builtin_amdgcn_perm(h.w, h.y, kLow), __builtin_amdgcn_perm(h.w, h.y, kHigh)};
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
// s + the sum of 8 bfloat16, in FP32 (products with 1 are exact).
__device__ __forceinline__ float add8(float s, u32x4 h) {
    const bf16x2 one = {(__bf16)1.f, (__bf16)1.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t two = h[i];
        s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, two), one, s, false);
    }
    return s;
}
// The sum of the four lanes l, l + 16, l + 32, l + 48, in all of them.
__device__ __forceinline__ float add_quarters(float s) {
    uint32_t u = __float_as_uint(s);
    auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    u = __float_as_uint(__uint_as_float(r[0]) + __uint_as_float(r[1]));
    r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Scales and zero points of one block of 128 k of a row, as they lie in
// memory (NS scales of 2 or 4 bytes, NS bytes).
template <int NS, int SB>
struct Groups {
    static constexpr int kWords = SB == 4 ? NS : (NS + 1) / 2;
    uint32_t s[kWords];
    uint32_t z;
};
template <int NS, int SB>
__device__ __forceinline__ float group_scale(const Groups<NS, SB>& g, int n, bool bf16) {
    if constexpr (SB == 4) return __uint_as_float(g.s[n]);
    const uint32_t raw = n % 2 ? g.s[n / 2] >> 16 : g.s[n / 2];
    const float f = (float)__builtin_bit_cast(_Float16, (uint16_t)raw);
    return bf16 ? __uint_as_float(raw << 16) : f;
}
// Drops the first sh groups (the same sh for the whole wave).
template <int NS, int SB>
__device__ __forceinline__ void end_groups(Groups<NS, SB>& g, int sh) {
    g.z >>= 8 * sh;
    if constexpr (SB == 4) {
        for (; sh > 0; --sh)
#pragma unroll
            for (int n = 0; n + 1 < NS; ++n) g.s[n] = g.s[n + 1];
    } else if constexpr (NS == 2) {
        g.s[0] >>= 16 * sh;
    } else {
        const uint64_t v = (((uint64_t)g.s[1] << 32) | g.s[0]) >> (16 * sh);
        g.s[0] = (uint32_t)v;
        g.s[1] = (uint32_t)(v >> 32);
    }
}

// NS values of T from p, at any alignment, into the low bytes of words.
template <int BYTES>
__device__ __forceinline__ void load_bytes(uint32_t* dst, const char* p) {
    if constexpr (BYTES == 1) {
        dst[0] = *reinterpret_cast<const uint8_t*>(p);
    } else if constexpr (BYTES == 2) {
        uint16_t v;
        __builtin_memcpy(&v, p, 2);
        dst[0] = v;
    } else {
        __builtin_memcpy(dst, p, BYTES);
    }
}

template <int NB, int MR, int SUB, int SB, bool CHUNKED>
__device__ __forceinline__ void quant_body(const QuantArgs& a, const QuantPlan& pl,
                                           int group_blocks) {
    extern __shared__ __align__(16) char smem[];
    constexpr int NS = 4 / SUB;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, q = lane >> 4;
    const int col0 = blockIdx.y * (16 * NB);
    const int ng = a.d / a.group;
    const int nks = a.d / 8;   // pieces of 8 k
    const int nmb = (a.V + 15) / 16;
    const int RW = kQWaves / pl.ksplit, rw = wave / pl.ksplit, kw = wave % pl.ksplit;
    // pass p of all workgroups sweeps one region of W, per_pass blocks each
    const int per_pass = pl.per_pass;
    const int ntile = (nmb + per_pass - 1) / per_pass;
    const int npass = (ntile - (int)blockIdx.x + pl.G - 1) / pl.G;
    auto block_of = [&](int pass, int m) {
        return ((int)blockIdx.x + pass * pl.G) * per_pass + m * RW + rw;
    };

    // this wave's k blocks of every pass
    const int kper = pl.nkb / pl.ksplit;
    const int kfirst = kw * kper;
    const bool has_zero = a.zero != nullptr;
    const bool scale_bf16 = a.scale_dtype == FS_BF16;
    const int row_bytes = a.d / 2;
    const char* zp = reinterpret_cast<const char*>(a.zero);

    // ---- W loader: k blocks of a pass in order, kQDepth of them ahead, two
    // at a time (a row's two neighbours share a 128-byte line)
    int ld_pass = 0, ld_k = 0;
    const char* qrow[MR];
    auto row_of = [&](int pass, int m, int r) {
        // rows past V re-read row V - 1 (not stored)
        return min(block_of(pass, m) * 16 + r, a.V - 1);
    };
    auto rows_of = [&](int pass) {
#pragma unroll
        for (int m = 0; m < MR; ++m)
            qrow[m] = reinterpret_cast<const char*>(a.q) +
                      (size_t)row_of(pass, m, r16) * row_bytes;
    };
    u32x4 w[kQDepth][MR];
    auto load = [&](u32x4 (&d0)[MR], u32x4 (&d1)[MR]) __attribute__((always_inline)) {
        const int o0 = (kfirst + ld_k) * 64 + q * 16;
        const int c0 = min(o0, row_bytes - 16), c1 = min(o0 + 64, row_bytes - 16);
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            d0[m] = __builtin_nontemporal_load((const global_u32x4*)(qrow[m] + c0));
            d1[m] = __builtin_nontemporal_load((const global_u32x4*)(qrow[m] + c1));
        }
        ld_k += 2;
        if (ld_k == kper) {
            ld_k = 0;
            if (ld_pass + 1 < npass) rows_of(++ld_pass);
        }
    };

    // ---- scales and zero points of kQDepth k blocks: lane (row, block) loads
    // the NS groups of one block of one row; they pass through the wave's own
    // LDS as pairs (s, -(16 + z)), [row block][block][group][row], which the
    // four quarters of the operand layout read back
    constexpr int kSlots = pair_slots(NB, NS);
    const int srow = lane >> 2, skb = lane & 3;
    float2* const pairs = reinterpret_cast<float2*>(smem + pl.pair_off) +
                          wave * (pl.mr * kSlots * NS * 16);
    int sc_pass = 0, sc_k = 0;
    Groups<NS, SB> graw[MR];
    auto load_scales = [&]() __attribute__((always_inline)) {
        const int kb = kfirst + sc_k + skb;
        // where the row ends inside the block, the row's last NS groups
        const int i = min(SUB == 4 ? kb / group_blocks : kb * NS, ng - NS);
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            const size_t at = (size_t)row_of(sc_pass, m, srow) * ng + i;
            load_bytes<NS * SB>(graw[m].s, static_cast<const char*>(a.scale) + at * SB);
            graw[m].z = 0x08080808u;
            if (has_zero) load_bytes<NS>(&graw[m].z, zp + at);
        }
    };
    // (of the blocks from..from + kSlots - 1 of the kQDepth)
    auto store_scales = [&](int from) __attribute__((always_inline)) {
        const int sh = (kfirst + sc_k + skb) * NS - (ng - NS);
        const int slot = skb - from;
        if (kSlots == kQDepth || (slot >= 0 && slot < kSlots)) {
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            if constexpr (NS > 1)
                if (sh > 0 && sh < NS) end_groups(graw[m], sh);
#pragma unroll
            for (int n = 0; n < NS; ++n)
                pairs[((m * kSlots + slot) * NS + n) * 16 + srow] =
                    make_float2(group_scale(graw[m], n, scale_bf16),
                                -16.f - (float)((graw[m].z >> (8 * n)) & 0xFFu));
        }
        }
        if (from + kSlots < kQDepth) return;
        sc_k += kQDepth;
        if (sc_k == kper) {
            sc_k = 0;
            if (sc_pass + 1 < npass) ++sc_pass;
        }
    };

    // ---- H: one (k block, 16 columns) unit per wave at a time
    const int nunits = pl.KC * NB;
    auto load_unit = [&](int chunk, int u, u32x4 (&h)[4]) {
        const int kb = chunk * pl.KC + u / NB;
        const int col = min(col0 + (u % NB) * 16 + r16, a.B - 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = kb * 16 + i * 4 + q;
            h[i] = p < nks ? *reinterpret_cast<const u32x4*>(a.H + (size_t)col * a.d + p * 8)
                           : u32x4{0u, 0u, 0u, 0u};
        }
    };
    auto store_unit = [&](char* buf, int u, const u32x4 (&h)[4]) {
        const int kb = u / NB, col = (u % NB) * 16 + r16;
        float* hs = reinterpret_cast<float*>(buf + pl.h_bytes);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // piece i * 4 + q: its step and quarter
            const int step = SUB == 4 ? q : SUB == 1 ? i : (i >> 1) * 2 + (q & 1);
            const int qq = SUB == 4 ? i : SUB == 1 ? q : (i & 1) + (q >> 1) * 2;
            if (col < pl.C)
                *reinterpret_cast<u32x4*>(buf + (((kb * 4 + step) * 4 + qq) * pl.C + col) * 16) =
                    permute_h(h[i]);
        }
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < SUB; ++i) s = add8(s, h[n * SUB + i]);
            s = add_quarters(s);
            if (q == 0) hs[(kb * NS + n) * (16 * NB) + col] = s;
        }
    };

    f32x4 total[MR][NB];
    // LDS offsets of this lane: its operand piece (columns past the stored
    // ones read the last: their results are not stored) and its sums.  One
    // block of k is at kb * 256 C, and kb * 64 NB NS.
    const int frag0 = (q * pl.C + min(r16, pl.C - 1)) * 16;
    const int frag_step = CHUNKED || NB > 1 ? 64 * 16 * NB : 64 * pl.C;   // one MFMA step
    const int sums0 = (int)pl.h_bytes + q * 16;
    // (the masks of unpack_word in registers, so that it is a shift and an
    // and-or)
    uint32_t nib_mask = 0x00780078u, sixteen = 0x41804180u;
    asm volatile("" : "+s"(nib_mask), "+v"(sixteen));
    // Two blocks of k: eight matrix steps, their LDS operands read kAheadH steps
    // before use, matrix and vector instructions in turn.
    auto consume = [&](int buf, int kb_lds, int slot, const u32x4 (&w0)[MR],
                       const u32x4 (&w1)[MR]) __attribute__((always_inline)) {
        constexpr int kSteps = 8;
        constexpr int kAheadH = NB == 1 ? 3 : NB == 2 ? 2 : 1;   // a step's latency to hide
        constexpr int kBufs = kAheadH + 1;
        u32x4 wt[2][MR];
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            wt[0][m] = transpose_words<SUB>(w0[m]);
            wt[1][m] = transpose_words<SUB>(w1[m]);
        }
        uint32_t frag = buf + frag0 + kb_lds * 4 * frag_step;
        uint32_t sums = buf + sums0 + kb_lds * (64 * NB * NS);
        asm volatile("" : "+v"(frag), "+v"(sums));   // one address each, formed here
        bf16x8 hf[kBufs][NB];
        f32x4 hsum[2][NB];
        float2 sc[2][MR];
        auto group_of = [](int st) { return st / SUB; };
        auto read = [&](int st) __attribute__((always_inline)) {
#pragma unroll
            for (int c = 0; c < NB; ++c)
                hf[st % kBufs][c] =
                    *reinterpret_cast<const bf16x8*>(smem + frag + st * frag_step + c * 256);
            if (st % SUB == 0) {
                const int g = group_of(st);
#pragma unroll
                for (int c = 0; c < NB; ++c)
                    hsum[g % 2][c] =
                        *reinterpret_cast<const f32x4*>(smem + sums + (g * NB + c) * 64);
#pragma unroll
                for (int m = 0; m < MR; ++m)
                    sc[g % 2][m] =
                        pairs[((m * kSlots + slot + g / NS) * NS + g % NS) * 16 + r16];
            }
        };
        // (hsum and sc hold two groups, the one in use and the next)
        constexpr int kAhead = kAheadH < SUB ? kAheadH : SUB;
#pragma unroll
        for (int st = 0; st < kAhead; ++st) read(st);
        f32x4 acc[MR][NB];
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
            if (st + kAhead < kSteps) read(st + kAhead);
            const int g = group_of(st);
            if (st % SUB == 0)
#pragma unroll
                for (int c = 0; c < NB; ++c)
#pragma unroll
                    for (int m = 0; m < MR; ++m) acc[m][c] = hsum[g % 2][c] * sc[g % 2][m].y;
            bf16x8 wf[MR];
#pragma unroll
            for (int m = 0; m < MR; ++m)
                wf[m] = unpack_word(wt[st / 4][m][st % 4], nib_mask, sixteen);
#pragma unroll
            for (int c = 0; c < NB; ++c)
#pragma unroll
                for (int m = 0; m < MR; ++m)
                    acc[m][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hf[st % kBufs][c], wf[m],
                                                                        acc[m][c], 0, 0, 0);
            if (st % SUB == SUB - 1)
#pragma unroll
                for (int c = 0; c < NB; ++c)
#pragma unroll
                    for (int m = 0; m < MR; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            total[m][c][i] = fmaf(sc[g % 2][m].x, acc[m][c][i], total[m][c][i]);
                            // here, not after the next loads (acc would stay alive)
                            asm volatile("" : "+v"(total[m][c][i]));
                        }
        }
        constexpr int kPer = 8 / NB + 2 * NS + 1;   // vector instructions per matrix one
#pragma unroll
        for (int st = -kAhead; st < kSteps; ++st) {
            if (st + kAhead < kSteps) {
                if ((st + kAhead) % SUB == 0)
                    __builtin_amdgcn_sched_group_barrier(0x100, 2 * NB + (MR + 1) / 2, 0);
                else
                    __builtin_amdgcn_sched_group_barrier(0x100, NB, 0);
            }
            if (st < 0) continue;
#pragma unroll
            for (int i = 0; i < NB * MR; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, kPer, 0);
            }
        }
    };
    // kQDepth blocks of k, from block k of the chunk at `buf`
    auto sweep = [&](int buf, int k) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kQDepth; i += 2) {
            if (i % kSlots == 0) {
                store_scales(i);
                if (i + kSlots == kQDepth) load_scales();
                // the wave's other lanes read them (LDS keeps a wave's order)
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
                __builtin_amdgcn_sched_barrier(0);
            }
            consume(buf, k + i, i % kSlots, w[i], w[i + 1]);
            __builtin_amdgcn_sched_barrier(0);
            load(w[i], w[i + 1]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto clear = [&]() {
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
            for (int c = 0; c < NB; ++c) total[m][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    };
    auto store = [&](int pass) {
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            const int row = block_of(pass, m) * 16 + r16;
            if (m * RW + rw >= per_pass || row >= a.V) continue;
#pragma unroll
            for (int c = 0; c < NB; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int b = col0 + c * 16 + q * 4 + i;
                    if (b < a.B) a.logits[(size_t)b * a.V + row] = total[m][c][i];
                }
        }
    };

    // ---- prologue: the first W blocks in flight, the first chunk of H in LDS
    rows_of(0);
#pragma unroll
    for (int i = 0; i < kQDepth; i += 2) load(w[i], w[i + 1]);
    load_scales();
    for (int u = wave; u < nunits; u += kQWaves) {
        u32x4 h[4];
        load_unit(0, u, h);
        store_unit(smem, u, h);
    }
    __syncthreads();

    if constexpr (!CHUNKED) {
        // ksplit > 1: the totals of a row block's waves meet in LDS, in the
        // order of k; each wave adds up and stores its share of the MR NB
        // (row block, column block) tiles.  Two areas, so that one barrier a
        // pass is enough.
        f32x4* red = reinterpret_cast<f32x4*>(smem + pl.h_bytes + pl.s_bytes);
        for (int pass = 0; pass < npass; ++pass) {
            clear();
            for (int k = kfirst; k < kfirst + kper; k += kQDepth) sweep(0, k);
            if (pl.ksplit == 1) {
                store(pass);
                continue;
            }
            f32x4* area = red + (pass & 1) * (kQWaves * MR * NB * 64);
#pragma unroll
            for (int m = 0; m < MR; ++m)
#pragma unroll
                for (int c = 0; c < NB; ++c)
                    area[((m * NB + c) * kQWaves + wave) * 64 + lane] = total[m][c];
            __syncthreads();
            const float* sums = reinterpret_cast<const float*>(area);
            for (int v = kw; v < MR * NB * 4; v += pl.ksplit) {   // value v % 4 of tile v / 4
                const int t = v >> 2, i = v & 3;
                const float* at = sums + ((t * kQWaves + rw * pl.ksplit) * 64 + lane) * 4 + i;
                float sum = at[0];
                for (int o = 1; o < pl.ksplit; ++o) sum += at[o * 256];
                const int row = block_of(pass, t / NB) * 16 + r16;
                const int b = col0 + t % NB * 16 + q * 4 + i;
                if (row < a.V && b < a.B) a.logits[(size_t)b * a.V + row] = sum;
            }
        }
    } else {
        const int step = (int)(pl.h_bytes + pl.s_bytes);
        int buf = 0;
        for (int pass = 0; pass < npass; ++pass) {
            clear();
            for (int c = 0; c < pl.nchunks; ++c) {
                const int other = step - buf;
                const int next = c + 1 < pl.nchunks ? c + 1 : 0;
                const bool more = pl.nchunks > 1 && (c + 1 < pl.nchunks || pass + 1 < npass);
                // the next chunk comes in while this one is used (units of a
                // wave: two at most, KC NB <= 2 kQWaves)
                u32x4 h0[4], h1[4];
                if (more && wave < nunits) load_unit(next, wave, h0);
                if (more && wave + kQWaves < nunits) load_unit(next, wave + kQWaves, h1);
                for (int k = 0; k < pl.KC; k += kQDepth) sweep(buf, k);
                if (more && wave < nunits) store_unit(smem + other, wave, h0);
                if (more && wave + kQWaves < nunits) store_unit(smem + other, wave + kQWaves, h1);
                if (more) {
                    __syncthreads();
                    buf = other;
                }
            }
            store(pass);
        }
    }
}

template <int NB, int MR, int SUB, int SB, bool CHUNKED>
__global__ __launch_bounds__(kQThreads, 2) void quant_kernel(QuantArgs a, QuantPlan pl,
                                                             int group_blocks) {
    if constexpr (CHUNKED && MR > 1) {
        // the last waves of a pass may have fewer blocks
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        if ((MR - 1) * kQWaves + wave >= pl.per_pass) {
            quant_body<NB, MR - 1, SUB, SB, CHUNKED>(a, pl, group_blocks);
            return;
        }
    }
    quant_body<NB, MR, SUB, SB, CHUNKED>(a, pl, group_blocks);
}

constexpr size_t kQLds = 160 * 1024;

QuantPlan quant_plan(const QuantArgs& a, int cus) {
    QuantPlan p{};
    // four column blocks from 33 columns on (two would read W twice: B=64,
    // d=5120, V=152057 300 against 240 us)
    p.nb = a.B <= 16 ? 1 : a.B <= 32 ? 2 : 4;
    const int nkb = (a.d + kQBlock - 1) / kQBlock;
    const int ns = a.group >= 128 ? 1 : 128 / a.group;
    const int nmb = (a.V + 15) / 16;
    auto round_up = [](int x, int m) { return (x + m - 1) / m * m; };
    auto bytes = [&](int kc) {
        p.h_bytes = (size_t)kc * 256 * p.C;
        p.s_bytes = (size_t)kc * ns * 16 * p.nb * 4;
        return p.h_bytes + p.s_bytes;
    };
    p.C = p.nb == 1 ? a.B : 16 * p.nb;
    // waves along k (kQDepth blocks each at least).  With several row blocks a
    // wave as many as can be: rows lie d / 2 bytes apart, so the waves that
    // share them read longer runs of fewer rows (B=1, d=4096, V=151936: 72 us,
    // unsplit 82 us).  With fewer, as many as give each wave one row block: a
    // pass over W then ends in one step (V=32000: unsplit 18, split by 8 23 us;
    // V=4000: 14 and 7 us)
    const int waves = cus * kQWaves;
    p.ksplit = 1;
    while (p.ksplit < kQWaves && 2 * p.ksplit * kQDepth <= nkb &&
           (nmb > 2 * waves || 2 * p.ksplit * nmb <= waves))
        p.ksplit *= 2;
    p.nkb = round_up(nkb, kQDepth * p.ksplit);
    auto rest = [&](int mr) {   // scales, totals
        return (size_t)kQWaves * mr * (pair_slots(p.nb, ns) * ns * 16 * 8) +
               (p.ksplit > 1 ? (size_t)2 * kQWaves * mr * p.nb * 64 * 16 : 0);
    };
    p.mr = 1;
    p.chunked = p.nb == 4 || bytes(p.nkb) + rest(1) > kQLds;
    if (!p.chunked) {
        p.KC = p.nkb;
        p.nchunks = 1;
        p.lds = bytes(p.KC) + rest(1);
        p.pair_off = p.lds - (size_t)kQWaves * (pair_slots(p.nb, ns) * ns * 16 * 8);
        int occ = (int)(kQLds / p.lds);
        if (occ > 2) occ = 2;
        p.per_pass = kQWaves / p.ksplit;
        const int ntile = (nmb + p.per_pass - 1) / p.per_pass;
        p.G = ntile < cus * occ ? ntile : cus * occ;
    } else {
        if (p.nb == 1) p.nb = 2;   // (chunks are built for two column blocks or four)
        p.C = 16 * p.nb;
        p.ksplit = 1;
        p.mr = 2;
        p.KC = 2 * kQWaves / p.nb / kQDepth * kQDepth;
        p.nkb = round_up(nkb, p.KC);
        p.nchunks = p.nkb / p.KC;
        p.pair_off = (p.nchunks == 1 ? 1 : 2) * bytes(p.KC);
        p.lds = p.pair_off + rest(p.mr);   // at most 152 KiB (group 32)
        // as many passes as full ones take, of equal length
        const int full = kQWaves * p.mr;
        p.G = nmb < cus ? nmb : cus;
        const int npass = (nmb + p.G * full - 1) / (p.G * full);
        p.per_pass = (nmb + p.G * npass - 1) / (p.G * npass);
        const int ntile = (nmb + p.per_pass - 1) / p.per_pass;
        if (p.G > ntile) p.G = ntile;
    }
    p.grid_y = (a.B + 16 * p.nb - 1) / (16 * p.nb);
    return p;
}

template <int NB, int MR, int SUB, int SB, bool CHUNKED>
hipError_t launch(const QuantArgs& a, const QuantPlan& p, hipStream_t stream) {
    const hipError_t e =
        hipFuncSetAttribute(reinterpret_cast<const void*>(&quant_kernel<NB, MR, SUB, SB, CHUNKED>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, (int)kQLds);
    if (e != hipSuccess) return e;
    const int group_blocks = a.group >= kQBlock ? a.group / kQBlock : 1;
    hipLaunchKernelGGL((quant_kernel<NB, MR, SUB, SB, CHUNKED>), dim3(p.G, p.grid_y),
                       dim3(kQThreads), p.lds, stream, a, p, group_blocks);
    return hipGetLastError();
}

template <int NB, int MR, int SB, bool CHUNKED>
hipError_t launch_sub(const QuantArgs& a, const QuantPlan& p, hipStream_t stream) {
    return a.group == 32   ? launch<NB, MR, 1, SB, CHUNKED>(a, p, stream)
           : a.group == 64 ? launch<NB, MR, 2, SB, CHUNKED>(a, p, stream)
                           : launch<NB, MR, 4, SB, CHUNKED>(a, p, stream);
}

template <int NB, int MR, bool CHUNKED>
hipError_t launch_nb(const QuantArgs& a, const QuantPlan& p, hipStream_t stream) {
    return a.scale_dtype == FS_F32 ? launch_sub<NB, MR, 4, CHUNKED>(a, p, stream)
                                   : launch_sub<NB, MR, 2, CHUNKED>(a, p, stream);
}

// d below one block of 128: one thread per logit, w = s (q - z) in FP32.
__global__ __launch_bounds__(256) void quant_short_kernel(QuantArgs a) {
    const int ng = a.group > 0 && a.d > 0 ? a.d / a.group : 0;
    const size_t n = (size_t)a.B * a.V;
    for (size_t o = (size_t)blockIdx.x * 256 + threadIdx.x; o < n; o += (size_t)gridDim.x * 256) {
        const int b = (int)(o / a.V), j = (int)(o % a.V);
        const uint8_t* q = a.q + (size_t)j * (a.d / 2);
        const __bf16* h = reinterpret_cast<const __bf16*>(a.H) + (size_t)b * a.d;
        float total = 0.f;
        for (int g = 0; g < ng; ++g) {
            const size_t i = (size_t)j * ng + g;
            const float s = a.scale_dtype == FS_F32    ? static_cast<const float*>(a.scale)[i]
                            : a.scale_dtype == FS_BF16 ? (float)static_cast<const __bf16*>(a.scale)[i]
                                                       : (float)static_cast<const _Float16*>(a.scale)[i];
            const float z = a.zero ? (float)a.zero[i] : 8.f;
            float sum = 0.f;
            for (int k = g * a.group; k < (g + 1) * a.group; k += 2) {
                const uint32_t v = q[k / 2];
                sum = fmaf((float)(v & 15u) - z, (float)h[k], sum);
                sum = fmaf((float)(v >> 4) - z, (float)h[k + 1], sum);
            }
            total = fmaf(s, sum, total);
        }
        a.logits[o] = total;
    }
}

}  // namespace

hipError_t launch_quant(const QuantArgs& a, int cus, hipStream_t stream) {
    if (a.d < kQBlock) {
        const size_t wgs = ((size_t)a.B * a.V + 255) / 256;
        hipLaunchKernelGGL(quant_short_kernel, dim3(wgs < 65536 ? (unsigned)wgs : 65536u), dim3(256), 0,
                           stream, a);
        return hipGetLastError();
    }
    const QuantPlan p = quant_plan(a, cus);
    if (!p.chunked)
        return p.nb == 1 ? launch_nb<1, 1, false>(a, p, stream)
                         : launch_nb<2, 1, false>(a, p, stream);
    return p.nb == 2 ? launch_nb<2, 2, true>(a, p, stream) : launch_nb<4, 2, true>(a, p, stream);
}

}  // namespace fs
