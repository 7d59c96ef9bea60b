// paged_decode.cu -- attention of new tokens over the sparse graph, keys and
// values in the pages of a cache:
//     out = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q . k_j),  j in N(pos)
//
// Bound: every key and value row of a (token, cache head) is read once, by all
// query heads of its group together, so the work is HBM traffic: 2 D es bytes
// for 4 G D operations, G query heads to a cache head.  Everything below is
// there to keep the loads in flight.  16 rows of 4,096 keys (8 cache heads of 128
// columns, bf16) take 46 us, 5.8 TB/s; one of 131,072 keys 95 us, 5.7 TB/s; 48
// ragged ones in 8 bits (101 MB) 30 us, of which 8 are the start of the shares
// and the join (new inputs from call to call).
//
// A warp owns a run of one row's edges and gathers them tile by tile with
// cp.async: rows are addressed one by one (edge -> position -> page -> cache
// row), so that windows, distance links, CSR lists and pages of any size go
// the same way.  A ring of stages per warp holds the tiles in flight; the
// positions and pages of later tiles are fetched ahead of their copies.
//
// 16-bit and 8-bit caches: mma.sync m16n8k16, S = Q K^T and O += P V, with
// eight (or sixteen) query heads as rows.  The tensor work is a fifth of the
// time that the bytes take, so the shape wastes nothing that counts, and the
// warp needs no other warp.  The sums over d (of S) and the columns (of O) may
// be taken in any order, so a lane's fragment is whatever 16 bytes of a row it
// can load at once:
//   S: lane (g, t) = (lane / 4, lane % 4) multiplies 16-byte pieces t, t + 4, ... of
//      key g;  O: pieces g, g + 8, ... of the value rows 2t, 2t+1, 2t+8, 2t+9.
// P has 16 bits in the product; each eight heads have a product of their own,
// whose lower eight rows carry what the rounding of P left over (P = hi + lo,
// 2^-17), so that the output is as good as with 32-bit probabilities.
//   8-bit rows become fp16 exactly.  A query row is scaled by a power of two
// into fp16's range; a value row's scale goes into its weight, and the weights
// have a running maximum of their own, so that no choice of scales overflows or
// loses them.  It goes in by its logarithm, weight = 2^(score + log2 scale - max):
// one exponential instead of a product whose range fp16 lacks, at the price of the
// logarithm's 2^-22 of its size (2^-19 of the weight for scales around 2^-10, 2^-15 at
// 2^-149), which the output's rounding by 2^-8 covers.
//
// fp32 caches: CUDA cores, a lane per key for the scores, a lane per four
// columns for the values, both from the staged tile.
//
// Two ways to share the work:
//   direct  rows that the graph keeps short: a CTA per (token, cache head), its
//           warps take equal runs and merge in shared memory.
//   split   the tiles of all rows, end to end, are cut into equal runs for all
//           warps of the GPU, wherever rows begin or end.  Whole rows are
//           finished by their warp; rows that are cut leave (m, l, acc), which
//           a second small kernel joins.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gather_common.cuh"
#include "paged_common.cuh"

namespace {

using namespace gather;

constexpr unsigned kFull = 0xffffffffu;

// ------------------------------------------------------------------ pieces

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}

// Copies of 4 or 16 bytes; with `on` false the bytes are set to zero and
// nothing is read.
template <int B>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, bool on) {
    const int n = on ? B : 0;
    if constexpr (B == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(B),
                     "r"(n)
                     : "memory");
}

__device__ __forceinline__ void copy_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copies_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 4, 8 or 16 bytes of shared memory.
template <int B>
__device__ __forceinline__ void load_words(uint32_t *w, uint32_t at) {
    if constexpr (B == 16)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(at));
    else if constexpr (B == 8)
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
    else
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at));
}

struct E4m3 {
    uint8_t x;
};

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1, __nv_bfloat16) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1, E4m3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t half_bits(__half2 h) {
    return *reinterpret_cast<uint32_t *>(&h);
}

// Four 8-bit values as fp16 ones (exact): bytes 0, 1 and bytes 2, 3.
__device__ __forceinline__ void widen(uint32_t four, uint32_t &lo, uint32_t &hi) {
    asm("{.reg .b16 x, y; mov.b32 {x, y}, %2; cvt.rn.f16x2.e4m3x2 %0, x; "
        "cvt.rn.f16x2.e4m3x2 %1, y;}"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}

// p0, p1 as 16-bit numbers and what their rounding leaves.
__device__ __forceinline__ void split16(float p0, float p1, uint32_t &hi, uint32_t &lo,
                                        __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    const __nv_bfloat162 r = __floats2bfloat162_rn(p0 - __uint_as_float(hi << 16),
                                                   p1 - __uint_as_float(hi & 0xffff0000u));
    lo = *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ void split16(float p0, float p1, uint32_t &hi, uint32_t &lo, E4m3) {
    const __half2 h = __floats2half2_rn(p0, p1);
    const float2 f = __half22float2(h);
    hi = half_bits(h);
    lo = half_bits(__floats2half2_rn(p0 - f.x, p1 - f.y));
}

// log2 of numbers down to fp32's smallest (the ftz form takes those below 2^-126 for zero).
__device__ __forceinline__ float lg2_any(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float finite_base(float m) { return m == -INFINITY ? 0.f : m; }

// --------------------------------------------------------------- arguments

// A row that a warp starts and others go on with: its first query head, the warp
// (of nw in a CTA), and its parts: `head` of them by warps of that CTA, then one
// from each of `mid` CTAs that have nothing else, then `tail` by the first warps
// of the next (head = 0: there is no such row).
struct __align__(16) Cut {
    int64_t nh;
    int32_t warp, head, mid, tail;
    int16_t gq, nw;
    __device__ __forceinline__ int count() const { return head + mid + tail; }
    // slot of part i
    __device__ __forceinline__ int64_t slot(int i) const {
        if (i < head) return 2 * ((int64_t)warp + i) + (i == 0 ? 1 : 0);
        const int cta = warp / nw + 1 + min(i - head, mid);
        return 2 * ((int64_t)cta * nw + max(i - head - mid, 0));
    }
};

struct DecodeArgs {
    const void *q, *k, *v;
    const float *k_scale, *v_scale;
    const int32_t *table, *row;
    const int64_t *pos;
    int64_t N, rows, max_pages, n_pages;
    int32_t H, Hkv, G, QB;  // query heads, cache heads, their ratio, blocks of it
    Divide page;
    float scale2;           // scale * log2(e)
    void *out;
    float *lse;
    float *part;  // partial rows [warp][2]: of the row it goes on with, of the one it starts
    Cut *cut;     // [warp]
    int *err;
};

// One token's row of edges.
struct Token {
    int64_t p;
    RowEdges e;
    const int32_t *pages;
    int32_t deg;
    bool bad;
};

__device__ __forceinline__ Token token_of(const DecodeArgs &a, const GraphView &g, int64_t n) {
    Token t;
    t.p = a.pos[n];
    const int64_t r = a.row ? a.row[n] : n;
    const bool ok = t.p >= 0 && t.p < g.T && t.p < a.max_pages * a.page.by && r >= 0 && r < a.rows;
    t.bad = !ok && t.p != -1;
    t.deg = 0;
    t.pages = a.table;
    t.e = RowEdges{};
    if (ok) {
        t.e = row_edges(g, t.p);
        t.deg = (int32_t)t.e.deg;
        t.pages = a.table + r * a.max_pages;
    }
    return t;
}

// A partial row: m[NQ], l[NQ], acc[NQ][D], fours of columns permuted within 32
// so that the lanes of a matrix product's result, eight columns and a row
// apart, meet different banks.
template <int NQ, int D>
struct Part {
    static constexpr int kHead = NQ < 2 ? 4 : 2 * NQ;  // (16-byte steps)
    static constexpr int kFloats = kHead + NQ * D;
    __device__ __forceinline__ static int place(int q, int four) {
        return kHead + q * D + 4 * (four ^ ((((four >> 3) << 1) | (q & 1)) & 7));
    }
};

// Joins two softmax states.
struct State {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ __forceinline__ void add(float m1, float l1, float4 o1) {
        const float mn = fmaxf(m, m1), base = finite_base(mn);
        const float w0 = ex2(m - base), w1 = ex2(m1 - base);
        l = l * w0 + l1 * w1;
        o.x = o.x * w0 + o1.x * w1;
        o.y = o.y * w0 + o1.y * w1;
        o.z = o.z * w0 + o1.z * w1;
        o.w = o.w * w0 + o1.w * w1;
        m = mn;
    }
    __device__ __forceinline__ float lse() const {
        return l == 0.f ? -INFINITY : (finite_base(m) + lg2(l)) * kLn2;
    }
};

__device__ __forceinline__ float4 divided(float4 o, float l) {
    const float r = 1.f / l;
    if (l == 0.f) return make_float4(0.f, 0.f, 0.f, 0.f);
    return make_float4(o.x * r, o.y * r, o.z * r, o.w * r);
}

__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 o) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(o.x, o.y), y = __floats2bfloat162_rn(o.z, o.w);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&x),
                                               *reinterpret_cast<const uint32_t *>(&y));
}
__device__ __forceinline__ void store4(float *p, float4 o) { *reinterpret_cast<float4 *>(p) = o; }

// ------------------------------------------------- 16-bit and 8-bit tiles

// One warp's work on tiles of KT keys.  NB: blocks of eight query heads.
template <typename T, int kD, int NB>
struct MmaTile {
    using Out = __nv_bfloat16;
    static constexpr bool k8 = sizeof(T) == 1;
    static constexpr int D = kD, NQ = 8 * NB;
    static constexpr int RB = D * (int)sizeof(T);          // bytes of a row
    // Tiles of 8 KB (less for short rows), two or three of them in flight per
    // warp: 130 to 200 KB an SM, where 45 would cover the latency of an idle
    // memory.  Twelve warps where their registers suffice (64 bf16 columns: 253
    // us for 32 rows of 16-32K keys, eight warps 259; 128 8-bit ones spill: 33 us
    // for a ragged batch of 103 MB, eight warps 30).
    static constexpr int KT = RB == 256 ? 16 : 32;
    static constexpr bool kMany = NB == 1 ? D == 64 : D == 32;
    static constexpr int kStages = RB == 32 ? 4 : RB == 128 && kMany ? 2 : 3;
    static constexpr int kWarps = kMany ? 12 : 8;
    static constexpr int kOcc = D == 32 && NB == 1 ? 2 : 1;
    static constexpr int KP = RB / 4 < 16 ? RB / 4 : 16, KN = RB / 4 / KP;
    static constexpr int VP = RB / 8 < 16 ? RB / 8 : 16, VN = RB / 8 / VP;
    static constexpr int VE = VP / (int)sizeof(T);
    static constexpr int kScaleBytes = k8 ? 2 * KT * 4 : 0;
    static constexpr int kStageBytes = 2 * KT * RB + kScaleBytes;
    static constexpr int kOwnBytes = 0;  // beyond the stages
    static constexpr int KS = D / 16, NT = D / 8;

    int lane, g, t;
    uint32_t qf[KS][NB == 1 ? 2 : 4];
    float unit[NB];  // of a score, in base 2
    float m[NB], l[NB];
    float mw[NB];    // running maximum of the weights (8-bit values)
    float acc[NB][NT][4];

    __device__ __forceinline__ void begin(const DecodeArgs &a, void *, int64_t n, int64_t h0,
                                          int gq) {
        lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        constexpr int KE = KP / (int)sizeof(T);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const bool on = b * 8 + g < gq;
            const uint8_t *q = (const uint8_t *)a.q + 2 * D * (n * a.H + h0 + (on ? b * 8 + g : 0));
            uint32_t w[D / 8];
#pragma unroll
            for (int x = 0; x < D / 8; x += 4) {
                const int e = 2 * x;  // element within the lane's D / 4
                const uint4 u = *reinterpret_cast<const uint4 *>(
                    q + 2 * ((e / KE * 4 + t) * KE + e % KE));
                w[x] = on ? u.x : 0, w[x + 1] = on ? u.y : 0;
                w[x + 2] = on ? u.z : 0, w[x + 3] = on ? u.w : 0;
            }
            unit[b] = a.scale2;
            if constexpr (k8) {
                uint32_t top = 0;
#pragma unroll
                for (int x = 0; x < D / 8; ++x)
                    top = max(top, max((w[x] << 16) & 0x7fffffffu, w[x] & 0x7fff0000u));
                top = max(top, __shfl_xor_sync(kFull, top, 1));
                top = max(top, __shfl_xor_sync(kFull, top, 2));
                // the row's largest magnitude to 2^14 .. 2^15; what falls below
                // fp16's 2^-24 is 2^-39 of it
                const int ex = max((int)(top >> 23) - 127, -100);
                const float up = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
                unit[b] *= __uint_as_float((uint32_t)(127 - 14 + ex) << 23);
#pragma unroll
                for (int x = 0; x < D / 8; ++x)
                    w[x] = half_bits(__floats2half2_rn(__uint_as_float(w[x] << 16) * up,
                                                       __uint_as_float(w[x] & 0xffff0000u) * up));
            }
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                qf[s][b] = w[2 * s];
                qf[s][NB + b] = w[2 * s + 1];
            }
            m[b] = mw[b] = -INFINITY;
            l[b] = 0.f;
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) acc[b][x][y] = 0.f;
        }
    }

    // A staged tile has its rows one after the other, the eight 16-byte pieces
    // of each 128 bytes permuted so that the lanes that read together meet
    // different banks: piece p of key row r lies at p ^ 4 (r mod 2) (two
    // neighbouring rows are read together), of value row r at p ^ 2 (r / 2 mod
    // 4) (four rows, two apart).  Shorter rows share 128 bytes; there the keys
    // need no permutation, and 32-byte values have none.  The functions below
    // split the places into a lane's part and constants.
    static constexpr bool kKeysXor = RB >= 128, kValuesXor = RB >= 64;

    // Piece i of key 8 x + g for lane (g, t).
    __device__ __forceinline__ uint32_t key_lane() const {
        return (g * RB + t * KP) ^ (kKeysXor ? (g & 1) << 6 : 0);
    }
    __device__ __forceinline__ static uint32_t key_at(uint32_t lane_part, int x, int i) {
        return (lane_part ^ ((i & 1) << 6)) + (i >> 1) * 128 + x * 8 * RB;
    }
    // Piece i of value row 16 x + 8 (y / 2) + 2 t + y mod 2.
    __device__ __forceinline__ uint32_t value_lane() const {
        return KT * RB + 2 * t * RB + ((g * VP) ^ (kValuesXor ? t << 5 : 0));
    }
    __device__ __forceinline__ static uint32_t value_at(uint32_t lane_part, int x, int y, int i) {
        const uint32_t odd = RB == 64 ? (lane_part ^ ((y & 1) << 6)) : lane_part + (y & 1) * RB;
        return odd + i * 128 + (y >> 1) * 8 * RB + x * 16 * RB;
    }

    // Start the copies of a tile: at[] are the offsets of its rows in the
    // cache, in bytes, -1 for none.  A row's lanes are neighbours.
    __device__ __forceinline__ void copy(const DecodeArgs &a, uint8_t *stage, const int64_t *at,
                                         bool every) const {
        constexpr int L = RB / 16, R = 32 / L;
        // lane (h, sub): piece sub of row R x + h; R rows are 512 bytes
        const int ln = threadIdx.x & 31, sub = ln % L, h = ln / L;
        const uint32_t dst = smem_addr(stage);
        const uint8_t *k = (const uint8_t *)a.k + sub * 16, *v = (const uint8_t *)a.v + sub * 16;
        const uint32_t to = h * RB + sub * 16;
        const uint32_t kd = dst + (to ^ (kKeysXor ? (h & 1) << 6 : 0));
        const uint32_t vl = to ^ (RB == 128 ? (h >> 1) << 5 : RB == 64 ? ((h >> 1) & 3) << 5 : 0);
        auto vd = [&](int x) {
            const int f = RB == 256 ? (x & 3) << 5 : RB == 128 ? (x & 1) << 6 : 0;
            return dst + KT * RB + (vl ^ f) + x * 512;
        };
        if (every) {
#pragma unroll
            for (int x = 0; x < KT / R; ++x) {
                const int64_t o = at[x * R + h];
                copy_async16(kd + x * 512, k + o);
                copy_async16(vd(x), v + o);
            }
        } else {
#pragma unroll 1
            for (int x = 0; x < KT / R; ++x) {
                const int64_t o = at[x * R + h];
                copy_async<16>(kd + x * 512, k + (o < 0 ? 0 : o), o >= 0);
                copy_async<16>(vd(x), v + (o < 0 ? 0 : o), o >= 0);
            }
        }
        if constexpr (k8) {
            const uint32_t sdst = dst + 2 * KT * RB;
#pragma unroll
            for (int x = 0; x < 2 * KT; x += 32) {
                const int i = x + ln;
                const int64_t o = at[i % KT];
                copy_async<4>(sdst + 4 * i, (i < KT ? a.k_scale : a.v_scale) + (o < 0 ? 0 : o / RB),
                              o >= 0);
            }
        }
    }

    __device__ __forceinline__ void tile(uint8_t *stage, uint32_t mask) {
        constexpr int KB = KT / 8;
        const uint32_t keys = smem_addr(stage) + key_lane();
        const uint32_t values = smem_addr(stage) + value_lane();
        float s[KB][4];
        float *scales = reinterpret_cast<float *>(stage + 2 * KT * RB);
        // The value scales' logarithms in their place, a lane for each (by every lane that
        // needs them: 32 rows of 16-32K keys of 64 columns 92 us, 94 this way; of 128
        // 152, 149), and their signs.
        uint32_t signs = 0;
        if constexpr (k8) {
            static_assert(KT == 32, "a lane for each key");
            const float x = scales[KT + lane];
            scales[KT + lane] = lg2_any(fabsf(x));
            signs = __ballot_sync(kFull, signbit(x)) >> 2 * t;
        }
        // scores
#pragma unroll
        for (int x = 0; x < KB; ++x) {
            float s2[2][4] = {};  // two sums side by side: half the chain
            uint32_t w[KN * KP / 4];
#pragma unroll
            for (int i = 0; i < KN; ++i) load_words<KP>(w + i * KP / 4, key_at(keys, x, i));
#pragma unroll
            for (int y = 0; y < KS; ++y) {
                uint32_t qa[4];
                qa[0] = qf[y][0];
                qa[2] = qf[y][NB];
                qa[1] = NB == 1 ? 0 : qf[y][NB - 1];
                qa[3] = NB == 1 ? 0 : qf[y][2 * NB - 1];
                if constexpr (k8) {
                    uint32_t b0, b1;
                    widen(w[y], b0, b1);
                    mma(s2[y & 1], qa, b0, b1, T());
                } else {
                    mma(s2[y & 1], qa, w[2 * y], w[2 * y + 1], T());
                }
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) s[x][y] = s2[0][y] + s2[1][y];
        }
        const uint32_t all = KT == 32 ? kFull : (1u << KT) - 1;
        uint32_t ph[NB][KB], pl[NB][KB];
        if constexpr (k8) __syncwarp();  // the logarithms are there
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float top = m[b], topw = mw[b];
            float lv[KB][2];  // log2 of the value scales
#pragma unroll
            for (int x = 0; x < KB; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int key = x * 8 + 2 * t + y;
                    float z = s[x][2 * b + y] * unit[b];
                    if constexpr (k8) {
                        z *= scales[key];
                        lv[x][y] = scales[KT + key];
                    }
                    s[x][2 * b + y] = z;
                }
            if (mask != all) {
#pragma unroll
                for (int x = 0; x < KB; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        if (!((mask >> (x * 8 + 2 * t + y)) & 1)) {
                            s[x][2 * b + y] = -INFINITY;
                            if constexpr (k8) lv[x][y] = 0.f;
                        }
            }
#pragma unroll
            for (int x = 0; x < KB; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    top = fmaxf(top, s[x][2 * b + y]);
                    if constexpr (k8) topw = fmaxf(topw, s[x][2 * b + y] + lv[x][y]);
                }
            top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
            top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
            const float base = finite_base(top);
            l[b] *= ex2(m[b] - base);
            float old = m[b], now = base;
            if constexpr (k8) {
                topw = fmaxf(topw, __shfl_xor_sync(kFull, topw, 1));
                topw = fmaxf(topw, __shfl_xor_sync(kFull, topw, 2));
                old = mw[b];
                now = finite_base(topw);
                mw[b] = topw;
            }
            const float fall = ex2(old - now);
            if (__any_sync(kFull, fall != 1.f)) {
#pragma unroll
                for (int x = 0; x < NT; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y) acc[b][x][y] *= fall;
            }
            m[b] = top;
#pragma unroll
            for (int x = 0; x < KB; ++x) {
                const float z0 = s[x][2 * b], z1 = s[x][2 * b + 1];
                float p0 = ex2(z0 - base), p1 = ex2(z1 - base);
                l[b] += p0 + p1;
                if constexpr (k8) {
                    // up to 2^14, so that fp16's smallest step is 2^-38 of the largest
                    p0 = ex2(z0 + lv[x][0] - now + 14.f);
                    p1 = ex2(z1 + lv[x][1] - now + 14.f);
                    p0 = __uint_as_float(__float_as_uint(p0) ^
                                         ((signs << (31 - 8 * x)) & 0x80000000u));
                    p1 = __uint_as_float(__float_as_uint(p1) ^
                                         ((signs << (30 - 8 * x)) & 0x80000000u));
                }
                split16(p0, p1, ph[b][x], pl[b][x], T());
            }
        }
        // values
#pragma unroll
        for (int x = 0; x < KT / 16; ++x)
#pragma unroll
            for (int i = 0; i < VN; ++i) {
                uint32_t w[4][VP / 4];
#pragma unroll
                for (int y = 0; y < 4; ++y) load_words<VP>(w[y], value_at(values, x, y, i));
#pragma unroll
                for (int z = 0; z < VP / 4; ++z) {
                    uint32_t b0[4], b1[4];
                    constexpr int E = k8 ? 4 : 2;
                    if constexpr (k8) {
                        widen(__byte_perm(w[0][z], w[1][z], 0x5140), b0[0], b0[1]);
                        widen(__byte_perm(w[0][z], w[1][z], 0x7362), b0[2], b0[3]);
                        widen(__byte_perm(w[2][z], w[3][z], 0x5140), b1[0], b1[1]);
                        widen(__byte_perm(w[2][z], w[3][z], 0x7362), b1[2], b1[3]);
                    } else {
                        b0[0] = __byte_perm(w[0][z], w[1][z], 0x5410);
                        b0[1] = __byte_perm(w[0][z], w[1][z], 0x7632);
                        b1[0] = __byte_perm(w[2][z], w[3][z], 0x5410);
                        b1[1] = __byte_perm(w[2][z], w[3][z], 0x7632);
                    }
#pragma unroll
                    for (int e = 0; e < E; ++e)
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            const uint32_t pa[4] = {ph[b][2 * x], pl[b][2 * x], ph[b][2 * x + 1],
                                                    pl[b][2 * x + 1]};
                            mma(acc[b][i * VE + z * E + e], pa, b0[e], b1[e], T());
                        }
                }
            }
    }

    // f(query, first column, four columns, m, l): the lane's share of the row.
    template <typename F>
    __device__ __forceinline__ void finish(F f) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            l[b] += __shfl_xor_sync(kFull, l[b], 1);
            l[b] += __shfl_xor_sync(kFull, l[b], 2);
            // The weights' unit, 2^(mw - 14 - m), by its square root, twice: value scales
            // reach from 2^-149 to 2^128, the unit goes below 2^-126.  (No weight at all:
            // the sums are zero.)
            const float back =
                !k8 ? 1.f : mw[b] == -INFINITY ? 0.f : ex2(0.5f * (mw[b] - 14.f - m[b]));
#pragma unroll
            for (int i = 0; i < VN; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int e = 0; e < VE; e += 4) {
                        float o[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float hi = acc[b][i * VE + e + y][c];
                            const float lo = acc[b][i * VE + e + y][2 + c];
                            // (an infinite value times a remainder of zero)
                            o[y] = fabsf(hi) < INFINITY ? hi + lo : hi;
                            if constexpr (k8) o[y] = o[y] * back * back;
                        }
                        f(b * 8 + g, (i * 8 + 2 * t + c) * VE + e,
                          make_float4(o[0], o[1], o[2], o[3]), m[b], l[b]);
                    }
        }
    }
};

// ------------------------------------------------------------ fp32 tiles

// The queries of a group are a constant (1, 2, 4, 8 or 16, the rest zero), so that
// their sums and shuffles run side by side.
template <int kD, int kNQ>
struct FmaTile {
    using Out = float;
    static constexpr int D = kD, NQ = kNQ, RB = 4 * D;
    static constexpr int KT = 1024 / D;   // 8 KB of keys and values
    // (a third stage where the queries leave room: 336 us instead of 393 for 16 rows
    // of 16-32K keys, D = 128, four heads to a group)
    static constexpr int kStages = NQ == 16 || (NQ == 8 && D == 128) ? 2 : 3;
    static constexpr int kWarps = 8, kOcc = 1;
    static constexpr int kStageBytes = 2 * KT * RB;
    static constexpr int kOwnBytes = NQ * D * 4 + NQ * KT * 4;  // queries and probabilities
    static constexpr int C = D / 4;       // 16-byte pieces of a row
    static constexpr int KG = 32 / C;     // keys side by side in the value sum
    static constexpr int KE = KT / KG;    // keys of a lane
    static_assert(KE == 8, "two groups of four");

    int lane;
    float *qs, *ps;
    float m[NQ], l[NQ];
    float4 acc[NQ];

    __device__ __forceinline__ void begin(const DecodeArgs &a, void *own, int64_t n, int64_t h0,
                                          int queries) {
        lane = threadIdx.x & 31;
        qs = (float *)own;
        ps = qs + NQ * D;
        __syncwarp();
        for (int x = lane; x < NQ * C; x += 32) {
            float4 q = make_float4(0.f, 0.f, 0.f, 0.f);  // (the queries beyond the group)
            if (x < queries * C)
                q = reinterpret_cast<const float4 *>((const float *)a.q + (n * a.H + h0) * D)[x];
            q.x *= a.scale2, q.y *= a.scale2, q.z *= a.scale2, q.w *= a.scale2;
            reinterpret_cast<float4 *>(qs)[x] = q;
        }
        __syncwarp();
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            m[x] = -INFINITY, l[x] = 0.f;
            acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }

    // Piece c of row r lies at place c ^ (r mod 8): eight lanes on eight rows
    // meet eight banks.
    __device__ __forceinline__ void copy(const DecodeArgs &a, uint8_t *stage, const int64_t *at,
                                         bool) const {
        const uint32_t dst = smem_addr(stage);
        const int ln = threadIdx.x & 31;
#pragma unroll
        for (int x = 0; x < KT * C; x += 32) {
            const int key = (x + ln) / C, c = (x + ln) % C;
            const int64_t o = at[key];
            const int64_t src = (o < 0 ? 0 : o) + c * 16;
            const uint32_t to = dst + key * RB + ((c ^ (key & 7)) << 4);
            copy_async<16>(to, (const uint8_t *)a.k + src, o >= 0);
            copy_async<16>(to + KT * RB, (const uint8_t *)a.v + src, o >= 0);
        }
    }

    __device__ __forceinline__ void tile(const uint8_t *stage, uint32_t mask) {
        const int key = lane % KT, part = lane / KT;  // 32 columns of a key
        float s[NQ];
#pragma unroll
        for (int x = 0; x < NQ; ++x) s[x] = 0.f;
#pragma unroll
        for (int c0 = 0; c0 < 8; ++c0) {
            // (parts two pieces apart: different banks for the queries)
            const int c = part * 8 + ((c0 + 2 * part) & 7);
            const float4 k =
                *reinterpret_cast<const float4 *>(stage + key * RB + ((c ^ (key & 7)) << 4));
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                const float4 q = reinterpret_cast<const float4 *>(qs)[x * C + c];
                s[x] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[x]))));
            }
        }
        const bool on = (mask >> key) & 1;
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            float z = s[x];
#pragma unroll
            for (int o = KT; o < 32; o <<= 1) z += __shfl_xor_sync(kFull, z, o);
            if (!on) z = -INFINITY;
            float top = z;
#pragma unroll
            for (int o = KT / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
            top = fmaxf(top, m[x]);
            const float base = finite_base(top), fall = ex2(m[x] - base);
            const float p = ex2(z - base);
            m[x] = top;
            l[x] = l[x] * fall + p;
            acc[x].x *= fall, acc[x].y *= fall, acc[x].z *= fall, acc[x].w *= fall;
            if (part == 0) ps[x * KT + key] = p;
        }
        __syncwarp();
        const int c = lane % C, kg = lane / C;
#pragma unroll
        for (int k0 = 0; k0 < KE; k0 += 4) {
            float4 v[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int j = kg * KE + k0 + y;
                v[y] = *reinterpret_cast<const float4 *>(stage + KT * RB + j * RB +
                                                         ((c ^ (j & 7)) << 4));
            }
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                const float4 p = *reinterpret_cast<const float4 *>(ps + x * KT + kg * KE + k0);
                const float pp[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    acc[x].x = fmaf(pp[y], v[y].x, acc[x].x);
                    acc[x].y = fmaf(pp[y], v[y].y, acc[x].y);
                    acc[x].z = fmaf(pp[y], v[y].z, acc[x].z);
                    acc[x].w = fmaf(pp[y], v[y].w, acc[x].w);
                }
            }
        }
        __syncwarp();
    }

    template <typename F>
    __device__ __forceinline__ void finish(F f) {
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
#pragma unroll
            for (int o = KT / 2; o; o >>= 1) l[x] += __shfl_xor_sync(kFull, l[x], o);
#pragma unroll
            for (int o = C; o < 32; o <<= 1) {
                acc[x].x += __shfl_xor_sync(kFull, acc[x].x, o);
                acc[x].y += __shfl_xor_sync(kFull, acc[x].y, o);
                acc[x].z += __shfl_xor_sync(kFull, acc[x].z, o);
                acc[x].w += __shfl_xor_sync(kFull, acc[x].w, o);
            }
            if (lane < C) f(x, 4 * lane, acc[x], m[x], l[x]);
        }
    }
};

// ------------------------------------------------------------- the kernels

template <typename Tile>
struct Layout {
    // per warp: the ring, what the tile type needs, the rows of the tile being
    // copied, the stages' masks
    static constexpr int kRing = Tile::kStages * Tile::kStageBytes;
    static constexpr int kRows = kRing + Tile::kOwnBytes;
    static constexpr int kMask = kRows + Tile::KT * 8;
    static constexpr int kBytes = (kMask + Tile::kStages * 4 + 127) / 128 * 128;
    using P = Part<Tile::NQ, Tile::D>;
    // (a warp's partial row of the direct way lies where its ring was)
    static_assert(P::kFloats * 4 <= kBytes, "a partial row fits a warp's storage");
    static_assert(kBytes * Tile::kWarps * Tile::kOcc <= 227 * 1024 - 4096 * Tile::kOcc, "smem");
};

// Query heads of block u of a token: first head and how many.
struct Block {
    int64_t kvh;
    int32_t first, gq;
};
template <int NQ>
__device__ __forceinline__ Block block_of(const DecodeArgs &a, int32_t u) {
    const int32_t kvh = u / a.QB, q0 = (u - kvh * a.QB) * NQ;
    return {kvh, kvh * a.G + q0, min(NQ, a.G - q0)};
}

// Edges [x0, x1) of a token's row for one block of query heads.
template <typename Tile>
__device__ __forceinline__ void run_edges(Tile &tile, const DecodeArgs &a, const GraphView &g,
                                          const Token &t, int64_t token, const Block &b, int32_t x0,
                                          int32_t x1, uint8_t *mem) {
    using M = Layout<Tile>;
    constexpr int S = Tile::kStages, KT = Tile::KT;
    const int lane = threadIdx.x & 31;
    int64_t *rows = reinterpret_cast<int64_t *>(mem + M::kRows);
    uint32_t *masks = reinterpret_cast<uint32_t *>(mem + M::kMask);
    const int32_t n = (x1 - x0 + KT - 1) / KT;
    const int32_t p = (int32_t)t.p, window = (int32_t)t.e.lo - t.e.ndil;

    constexpr uint32_t all = KT == 32 ? kFull : (1u << (KT & 31)) - 1;
    int32_t at = x0 + lane;      // the next edge of this lane to look up
    int32_t key = -1;            // its position
    int32_t page = -1, off = -1; // page and place of the one before
    auto next_key = [&] {
        key = -1;
        if (lane < KT && at < x1)
            key = g.kind != 0        ? g.colidx[t.e.start + at]
                  : at < t.e.ndil    ? p - (int32_t)g.offs[t.e.first + at]
                                     : window + at;
        at += KT;
    };
    auto next_page = [&] {
        page = off = -1;
        if (key >= 0) {
            const uint32_t x = divide((uint32_t)key, a.page);
            off = key - (int32_t)(x * a.page.by);
            page = t.pages[x];
        }
    };
    auto copy = [&](int stage) {
        const bool ok = off >= 0 && page >= 0 && page < a.n_pages;
        if (off >= 0 && !ok) atomicOr(a.err, SA_DEVERR_BOUNDS);
        const uint32_t mask = __ballot_sync(kFull, ok);
        __syncwarp();
        if (lane < KT)
            rows[lane] =
                ok ? (((int64_t)page * a.Hkv + b.kvh) * a.page.by + off) * Tile::RB : -1;
        if (lane == 0) masks[stage] = mask;
        __syncwarp();
        tile.copy(a, mem + stage * Tile::kStageBytes, rows, mask == all);
    };
    next_key();
    next_page();
    next_key();
    int stage = 0;
#pragma unroll
    for (int i = 0; i < S; ++i) {
        if (i < n) {
            copy(i);
            next_page();
            next_key();
        }
        copies_commit();
    }
    tile.begin(a, mem + M::kRing, token, b.first, b.gq);  // with the first copies under way
    // (the copies of a later tile come after the work on this one: in front they
    // would hold up its loads from shared memory)
    for (int32_t i = 0; i < n; ++i) {
        copies_wait<S - 1>();
        __syncwarp();
        tile.tile(mem + stage * Tile::kStageBytes, masks[stage]);
        __syncwarp();
        if (i + S < n) {
            copy(stage);
            next_page();
            next_key();
        }
        copies_commit();
        stage = stage + 1 == S ? 0 : stage + 1;
    }
    copies_wait<0>();
    __syncwarp();
}

template <typename Tile>
__device__ __forceinline__ void write_part(Tile &tile, float *slot) {
    constexpr int NQ = Tile::NQ, D = Tile::D;
    tile.finish([&](int q, int d, float4 o, float m, float l) {
        *reinterpret_cast<float4 *>(slot + Part<NQ, D>::place(q, d / 4)) = o;
        if (d == 0) slot[q] = m, slot[NQ + q] = l;
    });
}

// A row's output, or (with `to`) one part, from `count` parts by `threads`
// threads.  (Not inlined: code that runs once costs its fetch.)
template <typename Out, int NQ, int D>
__device__ __noinline__ void merge_parts(int tid, int threads, const float *const *part, int count,
                                         int gq, float *to, Out *out, float *lse) {
    constexpr int C = D / 4;
#pragma unroll 1
    for (int x = tid; x < gq * C; x += threads) {
        const int q = x / C, c = x % C;
        float m = -INFINITY, l = 0.f;
#pragma unroll 4
        for (int k = 0; k < count; ++k) m = fmaxf(m, part[k][q]);
        const float base = finite_base(m);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < count; ++k) {
            const float *p = part[k];
            const float w = ex2(p[q] - base);
            const float4 y = *reinterpret_cast<const float4 *>(p + Part<NQ, D>::place(q, c));
            l = fmaf(w, p[NQ + q], l);
            o.x = fmaf(w, y.x, o.x), o.y = fmaf(w, y.y, o.y);
            o.z = fmaf(w, y.z, o.z), o.w = fmaf(w, y.w, o.w);
        }
        if (to) {
            *reinterpret_cast<float4 *>(to + Part<NQ, D>::place(q, c)) = o;
            if (c == 0) to[q] = m, to[NQ + q] = l;
            continue;
        }
        store4(out + q * D + 4 * c, divided(o, l));
        if (c == 0) lse[q] = l == 0.f ? -INFINITY : (base + lg2(l)) * kLn2;
    }
}

// The direct way: CTA b has block b mod U of token b / U.
template <typename Tile>
__global__ void __launch_bounds__(32 * Tile::kWarps, Tile::kOcc)
    paged_decode_direct(DecodeArgs a, GraphView g) {
    using M = Layout<Tile>;
    extern __shared__ __align__(128) uint8_t mem[];
    __shared__ const float *s_part[Tile::kWarps];
    chain_begin();
    const int U = a.Hkv * a.QB, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int64_t n = blockIdx.x / U;
    const Block b = block_of<Tile::NQ>(a, blockIdx.x % U);
    const Token t = token_of(a, g, n);
    if (t.bad && threadIdx.x == 0) atomicOr(a.err, SA_DEVERR_BOUNDS);
    const int32_t tiles = (t.deg + Tile::KT - 1) / Tile::KT;
    const int32_t x0 = (int32_t)((int64_t)tiles * warp / nw) * Tile::KT;
    const int32_t x1 = min(t.deg, (int32_t)((int64_t)tiles * (warp + 1) / nw) * Tile::KT);
    uint8_t *own = mem + warp * M::kBytes;
    Tile tile;
    run_edges(tile, a, g, t, n, b, x0, x1, own);
    write_part(tile, (float *)own);
    if ((threadIdx.x & 31) == 0) s_part[warp] = (float *)own;
    __syncthreads();
    const int64_t nh = n * a.H + b.first;
    merge_parts<typename Tile::Out, Tile::NQ, Tile::D>(
        threadIdx.x, blockDim.x, s_part, nw, b.gq, nullptr,
        (typename Tile::Out *)a.out + nh * Tile::D, a.lse + nh);
}

// Equal shares of `total` tiles.
struct Shares {
    int64_t base, rem;
    __device__ Shares(int64_t total, int64_t n) : base(quotient(total, n)), rem(total - base * n) {}
    __device__ int64_t begin(int64_t w) const { return w * base + (w < rem ? w : rem); }
    __device__ int64_t of(int64_t x) const {
        const int64_t big = rem * (base + 1);
        return x < big ? quotient(x, base + 1) : rem + quotient(x - big, base);
    }
};

// What the start of a row costs a warp (positions, pages and the first copies
// one after the other, then its end), in tiles.  The shares count it: 40 ragged
// rows in 8 bits take 18 us, 24 if it counts 1, 19 if it counts 6; 100 ragged rows
// of 128 columns 56.5 us, 68 and 57.6.
constexpr int kRowStart = 3;
// Fewest tiles worth a warp: below, a share is mostly its own start (8 rows of
// 1,600 keys: 10.2 us, 10.7 with 4 or 8).
constexpr int kLeastTiles = 2;

template <typename Tile>
__global__ void __launch_bounds__(32 * Tile::kWarps, Tile::kOcc)
    paged_decode_split(DecodeArgs a, GraphView g) {
    using M = Layout<Tile>;
    constexpr int NW = Tile::kWarps, NT = 32 * NW, KT = Tile::KT;
    constexpr int PF = M::P::kFloats, D = Tile::D;
    using Out = typename Tile::Out;
    extern __shared__ __align__(128) uint8_t mem[];
    __shared__ int64_t s_start[NT + 1];  // what the rows before each thread's cost
    __shared__ int64_t s_sum[NW];
    __shared__ const float *s_part[NW];  // each warp's ring
    __shared__ int s_inside;             // queries of the row that has the whole CTA, or 0
    chain_begin();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t U = (int64_t)a.Hkv * a.QB;
    auto tiles_of = [&](int32_t deg) { return max(1, (deg + KT - 1) / KT); };
    auto cost_of = [&](int32_t deg) { return tiles_of(deg) + kRowStart; };

    // what all rows cost, and where each run of rows begins
    const int64_t per = (a.N + NT - 1) / NT;
    {
        int64_t own = 0;
        for (int64_t n = tid * per; n < min(a.N, (tid + 1) * per); ++n)
            own += cost_of(token_of(a, g, n).deg);
        int64_t x = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(kFull, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_sum[warp] = x;
        __syncthreads();
        for (int w = 0; w < warp; ++w) x += s_sum[w];
        s_start[tid + 1] = x;
        if (tid == 0) s_start[0] = 0, s_inside = 0;
        __syncthreads();
    }
    const int64_t total = s_start[NT] * U;
    const int64_t want = quotient(total, (int64_t)kLeastTiles * gridDim.x) + 1;
    const int nw = want < NW ? (int)want : NW;  // warps at work in each CTA
    const Shares shares(total, (int64_t)nw * gridDim.x);
    const int64_t W = (int64_t)blockIdx.x * nw + warp;
    int64_t x = warp < nw ? shares.begin(W) : 0;
    const int64_t x_end = warp < nw ? shares.begin(W + 1) : 0;
    uint8_t *own = mem + warp * M::kBytes;
    if (lane == 0) a.cut[blockIdx.x * NW + warp].head = 0;
    if (x < x_end) {
        // the row of tile x
        const int64_t y = quotient(x, U);
        int lo = -1;  // last run that begins at or before y
#pragma unroll
        for (int i = 0; i < NW; ++i) lo += __popc(__ballot_sync(kFull, s_start[32 * i + lane] <= y));
        int64_t n = lo * per, before = s_start[lo];
        if (per > 1) {
            for (;; n += 32) {
                const int64_t mine = n + lane;
                int64_t z = mine < a.N ? cost_of(token_of(a, g, mine).deg) : 0;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t up = __shfl_up_sync(kFull, z, o);
                    if (lane >= o) z += up;
                }
                const unsigned past = __ballot_sync(kFull, before + z > y);
                if (past || n + 32 >= a.N) {
                    const int f = past ? __ffs(past) - 1 : 31;
                    const int64_t b4 = __shfl_sync(kFull, z, f ? f - 1 : 0);
                    if (f) before += b4;
                    n += f;
                    break;
                }
                before += __shfl_sync(kFull, z, 31);
            }
        }
        n = min(n, a.N - 1);
        Token t = token_of(a, g, n);
        const int64_t in_row = x - before * U;
        int32_t tiles = tiles_of(t.deg);
        int32_t u = (int32_t)quotient(in_row, tiles + kRowStart);
        int32_t from = (int32_t)(in_row - (int64_t)u * (tiles + kRowStart));
        Tile tile;
        while (true) {
            // [from, to) of the row's cost; its first kRowStart are its start
            const int32_t to = (int32_t)min((int64_t)(tiles + kRowStart), from + (x_end - x));
            const int32_t tile0 = max(from - kRowStart, 0), tile1 = to - kRowStart;
            if (tile1 > 0) {
                if (t.bad && lane == 0) atomicOr(a.err, SA_DEVERR_BOUNDS);
                const Block b = block_of<Tile::NQ>(a, u);
                run_edges(tile, a, g, t, n, b, tile0 * KT, min(t.deg, tile1 * KT), own);
                const bool goes_on = tile0 > 0, ends = tile1 == tiles;
                write_part(tile, (float *)own);
                __syncwarp();
                const int64_t nh = n * a.H + b.first;
                // the row's first tile and its end, in the shares' coordinate
                const int64_t row0 = x - from + kRowStart, row1 = row0 + tiles;
                const bool inside = nw == NW && row0 < shares.begin(W - warp) &&
                                    row1 >= shares.begin(W - warp + nw);
                if (lane == 0) {
                    s_part[warp] = (const float *)own;
                    if (inside) s_inside = b.gq;
                }
                __syncwarp();
                if (!goes_on && ends) {
                    merge_parts<Out, Tile::NQ, D>(lane, 32, s_part + warp, 1, b.gq, nullptr,
                                                  (Out *)a.out + nh * D, a.lse + nh);
                } else if (!inside) {
                    float4 *part =
                        reinterpret_cast<float4 *>(a.part + (W * 2 + (goes_on ? 0 : 1)) * PF);
                    for (int i = lane; i < (M::P::kHead + b.gq * D) / 4; i += 32)
                        part[i] = reinterpret_cast<const float4 *>(own)[i];
                    if (!goes_on) {
                        const int64_t last = shares.of(row1 - 1), cta = quotient(last, nw);
                        // (CTAs of fewer warps merge nothing)
                        const int64_t next = nw < NW ? last + 1 : W - warp + nw;
                        Cut cut;
                        cut.nh = nh;
                        cut.warp = (int32_t)W;
                        cut.head = (int32_t)(min(last + 1, next) - W);
                        cut.mid = last < next ? 0 : (int32_t)cta - (int32_t)blockIdx.x - 1;
                        cut.tail = last < next ? 0 : (int32_t)(last + 1 - cta * nw);
                        if (cut.tail == NW && row1 == shares.begin(last + 1))
                            cut.tail = 0, ++cut.mid;  // nothing else in that CTA
                        cut.gq = (int16_t)b.gq;
                        cut.nw = (int16_t)nw;
                        if (lane == 0) a.cut[blockIdx.x * NW + warp] = cut;
                    }
                }
                __syncwarp();
            }
            x += to - from;
            if (x >= x_end) break;
            from = 0;
            if (++u == U) {
                u = 0;
                t = token_of(a, g, ++n);
                tiles = tiles_of(t.deg);
            }
        }
    }
    // a long row's parts in this CTA become one
    __syncthreads();
    if (s_inside)
        merge_parts<Out, Tile::NQ, D>(tid, NT, s_part, NW, s_inside,
                                      a.part + (int64_t)blockIdx.x * NW * 2 * PF, (Out *)nullptr,
                                      nullptr);
}

// The cut rows: block (c, q) joins query q of those that CTA c's warps start.
// The block's lane groups, a row of D columns each, are shared among them.
constexpr int kJoinThreads = 512;

template <typename Tile>
__global__ void __launch_bounds__(kJoinThreads) paged_decode_join(DecodeArgs a) {
    constexpr int NQ = Tile::NQ, D = Tile::D, C = D / 4, R = kJoinThreads / C, NW = Tile::kWarps;
    using P = Part<NQ, D>;
    static_assert(NW <= R && NW <= 32, "a group for each row");
    __shared__ Cut s_cut[NW];
    __shared__ int s_count;
    __shared__ float s_m[R], s_l[R];
    __shared__ float4 s_o[R][C];
    chain_begin();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        Cut cut = {};
        if (lane < NW) {
            const int4 *p = reinterpret_cast<const int4 *>(a.cut + blockIdx.x * NW + lane);
            int4 *to = reinterpret_cast<int4 *>(&cut);
            to[0] = __ldcg(p), to[1] = __ldcg(p + 1);
        }
        const unsigned there = __ballot_sync(kFull, cut.head > 0);
        if (cut.head > 0) s_cut[__popc(there & ((1u << lane) - 1))] = cut;
        if (lane == 0) s_count = __popc(there);
    }
    __syncthreads();
    if (s_count == 0) return;
    int each = R;  // groups of a row: a power of two
    while (each * s_count > R) each >>= 1;
    const int q = blockIdx.y, c = threadIdx.x % C, g = threadIdx.x / C;
    const int which = g / each, r = g % each;
    Cut cut = {};
    if (which < s_count) cut = s_cut[which];
    const int count = q < cut.gq ? cut.count() : 0;
    State s;
#pragma unroll 4
    for (int i = r; i < count; i += each) {
        const float *p = a.part + cut.slot(i) * P::kFloats;
        s.add(__ldcg(p + q), __ldcg(p + NQ + q),
              __ldcg(reinterpret_cast<const float4 *>(p + P::place(q, c))));
    }
    if (c == 0) s_m[g] = s.m, s_l[g] = s.l;
    s_o[g][c] = s.o;
    __syncthreads();
    if (r != 0 || count == 0) return;
#pragma unroll 4
    for (int i = g + 1; i < g + each; ++i) s.add(s_m[i], s_l[i], s_o[i][c]);
    const int64_t nh = cut.nh + q;
    store4((typename Tile::Out *)a.out + nh * D + 4 * c, divided(s.o, s.l));
    if (c == 0) a.lse[nh] = s.lse();
}

// ------------------------------------------------------------------- host

int64_t longest_row(const sa_graph_s *g) {
    int64_t n = g->kind == 0 ? (int64_t)g->W + g->n_off
                             : (int64_t)g->W + g->max_resid;
    return n < g->T ? n : g->T;
}

// Rows that the direct way takes, by the bytes of keys and values of the longest
// that the graph allows (the host does not know the positions).
//   Up to kDirectBytes it is the faster one for nearly every batch (direct and split,
// us: 8 rows of 128 KB 5.4, 9.0; of 384 KB 9.9, 10.2; of 512 KB 12.1, 10.5; 2,048
// rows of 128 KB 58, 56, of 384 KB 156, 139).
//   Up to kDirectSome where the rows are half to four times the SMs (160 bf16 rows of
// 768 KB 31, 33, 8-bit ones 43, 37; 512 rows 66, 77; 80 rows of 512 KB 20, 21).
//   Up to kDirectUniform on graphs of a window and up to 63 links, short of the
// sequences, where the rows fill the SMs in one go.  A CTA needs 17 us for a MB of
// 16-bit rows, 21 in fp32, 26 in 8 bits, the whole GPU 21 for 128 of them, and split
// 12 more for its shares and the join.  So it depends on the positions (112 to 144
// rows, D = 128, direct as a part of split's time):
//     whole windows   bf16 0.75-0.79 at 1 MB, 0.83-0.88 at 2.5, 0.86-0.90 at 4;
//                     fp32 0.76-0.79, 0.84-0.91, 0.87-0.96;  8 bits 0.84-0.87 at 1 MB,
//                     0.87-0.93 at 1.5, 0.96-1.05 at 4
//     from nothing to two windows, evenly   bf16 0.79-0.93, 0.88-1.06, 0.91-1.17;
//                     fp32 0.85-0.93, 1.01-1.14, 1.07-1.23;  8 bits 0.93-1.03, 1.02-1.13
//     one window, the others a sixteenth    bf16 1.5, 2.7, 3.7;  8 bits 1.9-2.1, 2.6
// The limit is where batches of the second kind come out even on average, 2.5 MB, or
// half of that in 8 bits; a batch of the third kind is slower by what one CTA takes for
// its row (48 us at 2.5 MB, 17 in shares).
constexpr int64_t kDirectBytes = 384 << 10, kDirectSome = 768 << 10, kDirectUniform = 2560 << 10;

int64_t longest_bytes(const sa_graph_s *g, const sa_paged_cache &c) {
    return longest_row(g) * 2 * c.D * (c.dtype == SA_FP32 ? 4 : c.dtype == SA_BF16 ? 2 : 1);
}

bool is_direct(const sa_graph_s *g, const sa_paged_cache &c, int64_t rows, int sms) {
    const int64_t bytes = longest_bytes(g, c);
    if (bytes <= kDirectBytes) return true;
    if (bytes <= kDirectSome && 2 * rows >= sms && rows <= 4 * sms) return true;
    const bool uniform = g->kind == 0 && g->W <= g->T / 4;
    return bytes <= (c.dtype == SA_E4M3 ? kDirectUniform / 2 : kDirectUniform) && uniform &&
           rows <= sms && 4 * rows >= 3 * sms;
}

// f(a Tile type) for this cache and group size.
template <typename F>
auto with_tile(const sa_paged_cache &c, int64_t G, F f)
    -> decltype(f((MmaTile<E4m3, 32, 1> *)0)) {
#define SA_PAGED_TILE(d)                                                              \
    if (c.D == d) {                                                                   \
        if (c.dtype == SA_BF16)                                                       \
            return G > 8 ? f((MmaTile<__nv_bfloat16, d, 2> *)0)                       \
                         : f((MmaTile<__nv_bfloat16, d, 1> *)0);                      \
        if (c.dtype == SA_E4M3)                                                       \
            return G > 8 ? f((MmaTile<E4m3, d, 2> *)0) : f((MmaTile<E4m3, d, 1> *)0); \
        return G > 8   ? f((FmaTile<d, 16> *)0)                                       \
               : G > 4 ? f((FmaTile<d, 8> *)0)                                        \
               : G > 2 ? f((FmaTile<d, 4> *)0)                                        \
               : G > 1 ? f((FmaTile<d, 2> *)0)                                        \
                       : f((FmaTile<d, 1> *)0);                                       \
    }
    SA_PAGED_TILE(32)
    SA_PAGED_TILE(64)
    SA_PAGED_TILE(128)
#undef SA_PAGED_TILE
    return {};
}

struct Plan {
    int64_t ctas = 0, part_floats = 0, warps = 0;
    size_t bytes() const {
        return ctas ? (size_t)(ctas * warps) * (2 * part_floats * 4 + sizeof(Cut)) : 0;
    }
};

template <typename Tile>
Plan split_plan(int sms) {
    Plan p;
    p.ctas = (int64_t)sms * Tile::kOcc;
    p.part_floats = Part<Tile::NQ, Tile::D>::kFloats;
    p.warps = Tile::kWarps;
    return p;
}

template <typename Tile>
sa_status launch_decode(DecodeArgs &a, const sa_graph_s *graph, const sa_paged_cache &cache,
                        void *workspace, cudaStream_t s) {
    using M = Layout<Tile>;
    a.QB = (a.G + Tile::NQ - 1) / Tile::NQ;
    const GraphView g = make_view(graph);
    const int64_t blocks = a.N * a.Hkv * a.QB, longest = longest_row(graph);
    int sms = 0;
    cudaError_t e = cudaSuccess;
    SA_CUDA_TRY(sa_sm_count(&sms));
    if (is_direct(graph, cache, blocks, sms)) {
        if (blocks > 0x7fffffffLL) return SA_ERR_UNSUPPORTED;
        // a warp for each tile, but only so many that all CTAs are on the GPU at
        // once: several of few warps overlap one's start with another's work (160
        // rows of 700 keys, D = 128: 15.4 us, 19.2 with eight warps in two turns)
        const int64_t per_sm = (blocks + sms - 1) / sms, held = Tile::kWarps * Tile::kOcc;
        int64_t nw = (longest + Tile::KT - 1) / Tile::KT;
        if (nw > held / per_sm) nw = held / per_sm;
        nw = nw < 1 ? 1 : nw > Tile::kWarps ? Tile::kWarps : nw;
        SA_CUDA_TRY(sa_smem_optin((const void *)paged_decode_direct<Tile>,
                                  Tile::kWarps * M::kBytes));
        SA_LAUNCH("paged_decode", s,
                  e = launch_chained(paged_decode_direct<Tile>, dim3((unsigned)blocks),
                                     32 * (int)nw, nw * M::kBytes, s, 1, a, g));
        SA_CUDA_TRY(e);
        return SA_OK;
    }
    const Plan p = split_plan<Tile>(sms);
    a.part = (float *)workspace;
    a.cut = (Cut *)(a.part + p.ctas * p.warps * 2 * p.part_floats);
    SA_CUDA_TRY(sa_smem_optin((const void *)paged_decode_split<Tile>, Tile::kWarps * M::kBytes));
    SA_LAUNCH("paged_decode", s,
              e = launch_chained(paged_decode_split<Tile>, dim3((unsigned)p.ctas),
                                 32 * Tile::kWarps, Tile::kWarps * M::kBytes, s, 1, a, g));
    SA_CUDA_TRY(e);
    const dim3 grid((unsigned)p.ctas, (unsigned)(a.G < Tile::NQ ? a.G : Tile::NQ));
    SA_LAUNCH("paged_decode_join", s,
              e = launch_chained(paged_decode_join<Tile>, grid, kJoinThreads, 0, s, 1, a));
    SA_CUDA_TRY(e);
    return SA_OK;
}

}  // namespace

size_t sa_paged_decode_workspace(const sa_tensor *q, const sa_paged_cache &c,
                                 const sa_graph_s *g) {
    int sms = 0;
    if (longest_bytes(g, c) <= kDirectBytes || sa_sm_count(&sms) != cudaSuccess) return 0;
    return with_tile(c, q->H / c.Hkv, [&](auto *t) {
        return split_plan<std::remove_pointer_t<decltype(t)>>(sms);
    }).bytes();
}

sa_status sa_paged_decode(const sa_tensor *q, const sa_paged_cache &c, const int32_t *table,
                          int64_t rows, int64_t max_pages, const int32_t *row, const int64_t *pos,
                          const sa_graph_s *g, float scale, sa_tensor *out, float *lse,
                          void *workspace, cudaStream_t s) {
    DecodeArgs a = {};
    a.q = q->ptr;
    a.k = c.k;
    a.v = c.v;
    a.k_scale = c.k_scale;
    a.v_scale = c.v_scale;
    a.table = table;
    a.row = row;
    a.pos = pos;
    a.N = q->B;
    a.rows = rows;
    a.max_pages = max_pages;
    a.n_pages = c.n_pages;
    a.H = (int32_t)q->H;
    a.Hkv = (int32_t)c.Hkv;
    a.G = (int32_t)(q->H / c.Hkv);
    a.page = make_divide((uint32_t)c.page_size);
    a.scale2 = scale * kLog2e;
    a.out = out->ptr;
    a.lse = lse;
    a.err = sa_device_error_word();
    if (!a.err) return SA_ERR_CUDA;
    struct Result {
        sa_status st = SA_ERR_UNSUPPORTED;
    };
    return with_tile(c, a.G, [&](auto *t) {
        return Result{launch_decode<std::remove_pointer_t<decltype(t)>>(
            a, g, c, workspace, s)};
    }).st;
}
