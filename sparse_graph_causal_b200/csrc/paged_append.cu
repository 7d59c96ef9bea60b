// paged_append.cu -- new key and value rows into the pages of a cache.
//
// Row t, head h goes to [slot / P, h, slot mod P, :].  A copy for bf16 and
// fp32; for an 8-bit cache every row gets its own scale:
//     scale = max_d |x_d| / 448,   code_d = e4m3(x_d / scale)
// Both divisions are IEEE fp32 ones, so that the largest value of a row is
// stored as exactly 448 and codes do not depend on how a product rounds.
//
// Bound: HBM, every row is read and written once (131,072 tokens of 8 heads of 128
// bf16 columns, 1.07 GB, 159 us: 6.7 TB/s, above a plain copy's 6.5, as some of the
// writes are still in L2 at the end); single tokens are bound by the chain slot ->
// page -> store (64 of them 3.3 us a call, 1.3 in a graph), the rounding by
// instructions (16,384 such tokens 19.4 us with new inputs, 16.2 with the inputs in
// L2, where the copy of their 102 MB would take 15.6).  A thread has kUnits 16-byte pieces of keys
// and as many of values, all loaded before the first slot is known.  The lanes
// of one row are neighbours (a power of two of them, 2 to 32), so that a row's
// largest magnitude is a few shuffles.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged_common.cuh"
#include "sa_internal.cuh"

namespace {

constexpr int kThreads = 256;

struct AppendArgs {
    const uint8_t *src[2];  // k, v
    int64_t stride[2];      // bytes from token to token
    uint8_t *dst[2];
    float *scale[2];
    const int64_t *slot;
    int64_t units;          // N * Hkv * L, pieces of each of k, v
    int64_t n_pages, Hkv;
    Divide per_token, page; // Hkv * L and P
    bool small;             // slots of the cache have 31 bits
    int *err;
};

// x / s, rounded to nearest but for quotients within 2^-45 of a border between
// two fp32 numbers, for 2^-60 <= s <= 2^60 (and x not far below; what is, has code
// 0): r is 1 / s rounded to nearest, x r is within 2^-23 of the quotient, and the
// correction by its remainder, itself off by 2^-23 of that, leaves 2^-45.  The
// quotients here are of bf16 numbers by 1 / 448 of one: none lies that close to a
// border that would change its code (checked over all pairs of significands), and
// amax / 448 is a seventh of a whole number of ulps away from every border, so that
// scales and codes are those of IEEE division.
__device__ __forceinline__ float quotient_rn(float x, float s, float r) {
    const float q = x * r;
    return fmaf(fmaf(-q, s, x), r, q);
}

// Two quotients as codes, the first in the low byte.
__device__ __forceinline__ uint32_t code4(float y0, float y1, float y2, float y3) {
    uint32_t c;
    asm("{.reg .b16 x, y; cvt.rn.satfinite.e4m3x2.f32 x, %2, %1; "
        "cvt.rn.satfinite.e4m3x2.f32 y, %4, %3; mov.b32 %0, {x, y};}"
        : "=r"(c)
        : "f"(y0), "f"(y1), "f"(y2), "f"(y3));
    return c;
}

// Scale and codes of a row in the ranges that the corrections do not cover
// (not inlined: hardly ever run).
__device__ __noinline__ float codes_by_division(float amax, const float *f, uint32_t *code) {
    const float scale = amax < INFINITY ? __fdiv_rn(amax, 448.f) : __uint_as_float(0x7fc00000u);
    for (int k = 0; k < 16; k += 4) {
        float y[4];
        for (int i = 0; i < 4; ++i) y[i] = scale > 0.f ? __fdiv_rn(f[k + i], scale) : 0.f;
        code[k / 4] = code4(y[0], y[1], y[2], y[3]);
    }
    return scale;
}

// Sixteen bf16 values of a row whose largest magnitude is amax (or NaN).
__device__ __forceinline__ uint4 codes(const uint4 (&x)[2], float amax, float &scale) {
    float f[16];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint4 &y = x[k / 4];
        const uint32_t b = k % 4 == 0 ? y.x : k % 4 == 1 ? y.y : k % 4 == 2 ? y.z : y.w;
        f[2 * k] = __uint_as_float(b << 16);
        f[2 * k + 1] = __uint_as_float(b & 0xffff0000u);
    }
    uint32_t c[4];
    if (amax >= 0x1p-50f && amax <= 0x1p60f) {
        scale = quotient_rn(amax, 448.f, 1.f / 448.f);
        const float r = __frcp_rn(scale);
#pragma unroll
        for (int k = 0; k < 16; k += 4)
            c[k / 4] = code4(quotient_rn(f[k], scale, r), quotient_rn(f[k + 1], scale, r),
                             quotient_rn(f[k + 2], scale, r), quotient_rn(f[k + 3], scale, r));
    } else {
        float g[16];
        uint32_t d[4];
        for (int k = 0; k < 16; ++k) g[k] = f[k];
        scale = codes_by_division(amax, g, d);
        for (int k = 0; k < 4; ++k) c[k] = d[k];
    }
    return make_uint4(c[0], c[1], c[2], c[3]);
}

// L: threads per row, of 16 bytes of input each (32 where they are rounded, so
// that the row's own work is shared by more values).
template <int L, bool kQuant, int kUnits>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const AppendArgs a) {
    const int64_t base = (int64_t)blockIdx.x * (kThreads * kUnits);
    const int64_t t0 = quotient(base, a.per_token.by);  // token of the block's first piece
    const uint32_t r0 = (uint32_t)(base - t0 * a.per_token.by);
    chain_begin();
    constexpr int V = kQuant ? 2 : 1;
    uint4 x[2][kUnits][V];
    int64_t token[kUnits];
    uint32_t piece[kUnits];
    int64_t slot[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const uint32_t u = i * kThreads + threadIdx.x;
        const uint32_t q = divide(r0 + u, a.per_token);
        token[i] = t0 + q;
        piece[i] = r0 + u - q * a.per_token.by;
        const bool in = base + u < a.units;
        slot[i] = in ? a.slot[token[i]] : -1;
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int y = 0; y < V; ++y)
                x[w][i][y] =
                    in ? reinterpret_cast<const uint4 *>(a.src[w] + token[i] * a.stride[w])
                             [piece[i] * V + y]
                       : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        bool ok = slot[i] >= 0;
        const uint32_t h = piece[i] / L, sub = piece[i] % L;
        int64_t dst = 0;  // row of the cache
        if (ok) {
            int64_t page, r;
            if (a.small && slot[i] <= 0x7fffffff) {
                page = divide((uint32_t)slot[i], a.page);
                r = (uint32_t)slot[i] - (uint32_t)page * a.page.by;
            } else {
                page = slot[i] / a.page.by;
                r = slot[i] - page * a.page.by;
            }
            if (page >= a.n_pages) {
                atomicOr(a.err, SA_DEVERR_BOUNDS);
                ok = false;
            }
            dst = (page * a.Hkv + h) * a.page.by + r;
        }
        if constexpr (!kQuant) {
            if (ok) {
                reinterpret_cast<uint4 *>(a.dst[0])[dst * L + sub] = x[0][i][0];
                reinterpret_cast<uint4 *>(a.dst[1])[dst * L + sub] = x[1][i][0];
            }
        } else {
            float top[2];  // largest magnitudes, NaN if there is one
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const __nv_bfloat162 *b = reinterpret_cast<const __nv_bfloat162 *>(&x[w][i][0]);
                __nv_bfloat162 m = __habs2(b[0]);
#pragma unroll
                for (int k = 1; k < 8; ++k) m = __hmax2_nan(m, __habs2(b[k]));
#pragma unroll
                for (int o = 1; o < L; o <<= 1)
                    m = __hmax2_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                top[w] = __bfloat162float(__hmax_nan(m.x, m.y));
            }
            if (ok) {
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    float scale;
                    const uint4 code = codes(x[w][i], top[w], scale);
                    reinterpret_cast<uint4 *>(a.dst[w])[dst * L + sub] = code;
                    if (sub == 0) a.scale[w][dst] = scale;
                }
            }
        }
    }
}

template <int L, bool kQuant, int kUnits>
sa_status launch_units(const AppendArgs &a, cudaStream_t s) {
    const int64_t blocks = (a.units + kThreads * kUnits - 1) / (kThreads * kUnits);
    if (blocks > 0x7fffffffLL) return SA_ERR_UNSUPPORTED;
    cudaError_t e = cudaSuccess;
    SA_LAUNCH("paged_append", s,
              e = launch_chained(paged_append_kernel<L, kQuant, kUnits>, dim3((unsigned)blocks),
                                 kThreads, 0, s, 1, a));
    SA_CUDA_TRY(e);
    return SA_OK;
}

// Four pieces a thread keep enough loads in flight (two where they are rounded:
// the code of four outgrows the instruction cache); few rows go one piece a
// thread, over more SMs.
constexpr int64_t kFewUnits = 148 * 4 * kThreads;

template <int L, bool kQuant>
sa_status launch_append(const AppendArgs &a, cudaStream_t s) {
    return a.units <= kFewUnits ? launch_units<L, kQuant, 1>(a, s)
                                : launch_units<L, kQuant, kQuant ? 2 : 4>(a, s);
}

}  // namespace

sa_status sa_paged_append(const sa_tensor *k, int64_t k_stride, const sa_tensor *v,
                          int64_t v_stride, const int64_t *slot, const sa_paged_cache &c,
                          cudaStream_t s) {
    const bool quant = c.dtype == SA_E4M3;
    const int es = k->dtype == SA_BF16 ? 2 : 4;
    const int L = (int)(c.D * es / (quant ? 32 : 16));
    AppendArgs a = {};
    a.src[0] = (const uint8_t *)k->ptr;
    a.src[1] = (const uint8_t *)v->ptr;
    a.stride[0] = k_stride * es;
    a.stride[1] = v_stride * es;
    a.dst[0] = (uint8_t *)c.k;
    a.dst[1] = (uint8_t *)c.v;
    a.scale[0] = c.k_scale;
    a.scale[1] = c.v_scale;
    a.slot = slot;
    a.units = k->B * c.Hkv * L;
    a.n_pages = c.n_pages;
    a.Hkv = c.Hkv;
    a.per_token = make_divide((uint32_t)(c.Hkv * L));
    a.page = make_divide((uint32_t)c.page_size);
    a.small = c.n_pages <= 0x7fffffffLL / c.page_size;
    a.err = sa_device_error_word();
    if (!a.err) return SA_ERR_CUDA;
    if (quant) switch (L) {
            case 2: return launch_append<2, true>(a, s);
            case 4: return launch_append<4, true>(a, s);
            case 8: return launch_append<8, true>(a, s);
        }
    else switch (L) {
            case 4: return launch_append<4, false>(a, s);
            case 8: return launch_append<8, false>(a, s);
            case 16: return launch_append<16, false>(a, s);
            case 32: return launch_append<32, false>(a, s);
        }
    return SA_ERR_UNSUPPORTED;
}
