// paged_append.cu -- new key and value rows into the pages of a cache.
//
// Row t, head h goes to [slot / P, h, slot mod P, :].  A copy for bf16 and
// fp32; for an 8-bit cache every row gets its own scale:
//     scale = max_d |x_d| / 448,   code_d = e4m3(x_d / scale)
// Both divisions are IEEE fp32 ones, so that the largest value of a row is
// stored as exactly 448 and codes do not depend on how a product rounds.  HBM
// bound: every row is read and written once, keys and values in one launch.
// A thread moves 16 bytes of input; the lanes of one row are neighbours (a
// power of two of them, 2 to 32), so that a row's largest magnitude is a few
// shuffles.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sa_internal.cuh"

namespace {

constexpr int kThreads = 256;

struct AppendArgs {
    const uint8_t *src[2];  // k, v
    int64_t stride[2];      // bytes from token to token
    uint8_t *dst[2];
    float *scale[2];
    const int64_t *slot;
    int64_t units;  // N * Hkv * L, threads needed for one of k, v
    int64_t n_pages;
    uint32_t Hkv, P;
    int *err;
};

// L: threads per row (16 bytes of input each).
template <int L, bool kQuant>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(AppendArgs a) {
    const int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int which = blockIdx.y;
    const bool in = u < a.units;
    const int sub = (int)(u % L);
    const int64_t rh = in ? u / L : 0;
    const int64_t t = rh / a.Hkv;
    const uint32_t h = (uint32_t)(rh - t * a.Hkv);
    const int64_t slot = in ? a.slot[t] : -1;
    bool ok = slot >= 0;
    int64_t dst = 0;  // row of the cache
    if (ok) {
        const int64_t page = slot / a.P, r = slot - page * a.P;
        if (page >= a.n_pages) {
            atomicOr(a.err, SA_DEVERR_BOUNDS);
            ok = false;
        }
        dst = (page * a.Hkv + h) * a.P + r;
    }
    uint4 x = make_uint4(0, 0, 0, 0);
    if (ok)
        x = __ldg(reinterpret_cast<const uint4 *>(a.src[which] + t * a.stride[which]) +
                  (h * L + sub));
    if (!kQuant) {
        if (ok) reinterpret_cast<uint4 *>(a.dst[which])[dst * L + sub] = x;
        return;
    }
    float f[8];
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    // the largest magnitude as an integer: bf16 magnitudes order like their
    // bits, and infinities and NaN stay on top
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[2 * k] = __uint_as_float(w[k] << 16);
        f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        top = max(top, max((w[k] << 16) & 0x7fffffffu, w[k] & 0x7fff0000u));
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (!ok) return;
    const float amax = __uint_as_float(top);
    const float scale = top < 0x7f800000u ? __fdiv_rn(amax, 448.f) : __uint_as_float(0x7fc00000u);
    uint32_t code[2] = {0, 0};
    if (scale > 0.f) {
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            const float2 y = make_float2(__fdiv_rn(f[k], scale), __fdiv_rn(f[k + 1], scale));
            const uint32_t c = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
            code[k / 4] |= c << (16 * ((k / 2) & 1));
        }
    }
    reinterpret_cast<uint2 *>(a.dst[which])[dst * L + sub] = make_uint2(code[0], code[1]);
    if (sub == 0) a.scale[which][dst] = scale;
}

template <int L, bool kQuant>
sa_status launch_append(const AppendArgs &a, cudaStream_t s) {
    const int64_t blocks = (a.units + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffLL) return SA_ERR_UNSUPPORTED;
    SA_LAUNCH("paged_append", s,
              paged_append_kernel<L, kQuant><<<dim3((unsigned)blocks, 2), kThreads, 0, s>>>(a));
    SA_CUDA_TRY(cudaGetLastError());
    return SA_OK;
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
    a.Hkv = (uint32_t)c.Hkv;
    a.P = (uint32_t)c.page_size;
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
