// paged_append.cu -- new key and value rows into the pages of a cache.
//
// Row t, head h goes to [slot / P, h, slot mod P, :].  A copy for bf16 and
// fp32; for an 8-bit cache every row gets its own scale:
//     scale = max_d |x_d| / 448,   code_d = e4m3(x_d / scale)
// Both divisions are IEEE fp32 ones, so that the largest value of a row is
// stored as exactly 448 and codes do not depend on how a product rounds.
//
// Bound: HBM, every row is read and written once; single tokens are bound by
// the chain slot -> page -> store.  A thread has kUnits 16-byte pieces of keys
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
    int64_t units;          // N * Hkv * L, 16-byte pieces of each of k, v
    int64_t n_pages, Hkv;
    Divide per_token, page; // Hkv * L and P
    bool small;             // slots of the cache have 31 bits
    int *err;
};

// Correctly rounded x / s for 2^-60 <= s <= 2^60 and quotients above 2^-40
// (smaller ones are off by less than 2^-60): r is 1 / s rounded to nearest,
// the first correction brings the quotient within an ulp, and by P. Markstein's
// theorem (IBM J. Res. Dev. 34, 1990) the second makes it the nearest.
__device__ __forceinline__ float quotient_rn(float x, float s, float r) {
    float q = x * r;
    q = fmaf(fmaf(-q, s, x), r, q);
    return fmaf(fmaf(-q, s, x), r, q);
}

// Eight bf16 values of a row whose largest magnitude has the bits `top`.
__device__ __forceinline__ uint2 codes(uint4 x, uint32_t top, float &scale) {
    const uint32_t b[4] = {x.x, x.y, x.z, x.w};
    scale = top < 0x7f800000u ? __fdiv_rn(__uint_as_float(top), 448.f)
                              : __uint_as_float(0x7fc00000u);
    uint32_t code[2] = {0, 0};
    if (scale > 0.f) {
        const bool plain = scale >= 0x1p-60f && scale <= 0x1p60f;
        const float r = __frcp_rn(scale);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float f0 = __uint_as_float(b[k] << 16);
            const float f1 = __uint_as_float(b[k] & 0xffff0000u);
            float2 y = make_float2(quotient_rn(f0, scale, r), quotient_rn(f1, scale, r));
            if (!plain) y = make_float2(__fdiv_rn(f0, scale), __fdiv_rn(f1, scale));
            const uint32_t c = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
            code[k / 2] |= c << (16 * (k & 1));
        }
    }
    return make_uint2(code[0], code[1]);
}

// L: threads per row (16 bytes of input each).
template <int L, bool kQuant, int kUnits>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const AppendArgs a) {
    const int64_t base = (int64_t)blockIdx.x * (kThreads * kUnits);
    const int64_t t0 = quotient(base, a.per_token.by);  // token of the block's first piece
    const uint32_t r0 = (uint32_t)(base - t0 * a.per_token.by);
    uint4 x[2][kUnits];
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
            x[w][i] = in ? __ldg(reinterpret_cast<const uint4 *>(a.src[w] + token[i] * a.stride[w]) +
                                 piece[i])
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
                reinterpret_cast<uint4 *>(a.dst[0])[dst * L + sub] = x[0][i];
                reinterpret_cast<uint4 *>(a.dst[1])[dst * L + sub] = x[1][i];
            }
        } else {
            // the largest magnitudes as integers: bf16 magnitudes order like
            // their bits, and infinities and NaN stay on top
            uint32_t top[2];
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const uint32_t b[4] = {x[w][i].x, x[w][i].y, x[w][i].z, x[w][i].w};
                top[w] = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    top[w] = max(top[w], max((b[k] << 16) & 0x7fffffffu, b[k] & 0x7fff0000u));
#pragma unroll
                for (int o = 1; o < L; o <<= 1)
                    top[w] = max(top[w], __shfl_xor_sync(0xffffffffu, top[w], o));
            }
            if (ok) {
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    float scale;
                    const uint2 code = codes(x[w][i], top[w], scale);
                    reinterpret_cast<uint2 *>(a.dst[w])[dst * L + sub] = code;
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
    SA_LAUNCH("paged_append", s,
              paged_append_kernel<L, kQuant, kUnits><<<(unsigned)blocks, kThreads, 0, s>>>(a));
    SA_CUDA_TRY(cudaGetLastError());
    return SA_OK;
}

// Four pieces a thread keep enough loads in flight; few rows go one piece a
// thread, over more SMs.
constexpr int64_t kFewUnits = 148 * 4 * kThreads;

template <int L, bool kQuant>
sa_status launch_append(const AppendArgs &a, cudaStream_t s) {
    return a.units <= kFewUnits ? launch_units<L, kQuant, 1>(a, s)
                                : launch_units<L, kQuant, 4>(a, s);
}

}  // namespace

sa_status sa_paged_append(const sa_tensor *k, int64_t k_stride, const sa_tensor *v,
                          int64_t v_stride, const int64_t *slot, const sa_paged_cache &c,
                          cudaStream_t s) {
    const bool quant = c.dtype == SA_E4M3;
    const int es = k->dtype == SA_BF16 ? 2 : 4;
    const int L = (int)(c.D * es / 16);
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
    switch (L) {
        case 4: return quant ? launch_append<4, true>(a, s) : launch_append<4, false>(a, s);
        case 8: return quant ? launch_append<8, true>(a, s) : launch_append<8, false>(a, s);
        case 16: return quant ? launch_append<16, true>(a, s) : launch_append<16, false>(a, s);
        case 32: return launch_append<32, false>(a, s);
    }
    return SA_ERR_UNSUPPORTED;
}
