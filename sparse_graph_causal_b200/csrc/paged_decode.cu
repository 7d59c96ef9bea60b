// paged_decode.cu -- attention of new tokens over the sparse graph, keys and
// values in the pages of a cache.
//
// One CTA per (token, query head): groups of lanes hold one cached row each
// (16 bytes per lane), every group has its own online-softmax state, merged
// by shuffles and then across the warps in shared memory.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gather_common.cuh"

namespace {

using namespace gather;

constexpr int kWarps = 8;

struct DecodeArgs {
    const void *q, *k, *v;
    const float *k_scale, *v_scale;
    const int32_t *table, *row;
    const int64_t *pos;
    int64_t rows, max_pages, n_pages;
    int32_t H, Hkv, P;
    float scale2;
    void *out;
    float *lse;
    int *err;
};

struct E4m3 {
    uint8_t x;
};

template <typename T>
struct Row {
    using Q = T;
    static constexpr int V = Slice<T>::V;
    __device__ static void load(const void *p, int64_t at, float *f) {
        Slice<T>::load((const T *)p + at, f);
    }
};
template <>
struct Row<E4m3> {
    using Q = __nv_bfloat16;
    static constexpr int V = 8;
    __device__ static void load(const void *p, int64_t at, float *f) {
        const __nv_fp8x4_e4m3 *x = (const __nv_fp8x4_e4m3 *)((const uint8_t *)p + at);
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const float4 y = (float4)x[a];
            f[4 * a] = y.x;
            f[4 * a + 1] = y.y;
            f[4 * a + 2] = y.z;
            f[4 * a + 3] = y.w;
        }
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps) paged_decode_kernel(DecodeArgs a, GraphView g) {
    using Q = typename Row<T>::Q;
    constexpr int V = Row<T>::V, L = D / V, G = 32 / L;
    constexpr int NG = G * kWarps;
    __shared__ float s_m[kWarps], s_l[kWarps];
    __shared__ float s_acc[kWarps][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int grp = lane / L, sub = lane % L;
    const int64_t nh = blockIdx.x, n = nh / a.H, h = nh % a.H;
    const int64_t kvh = h / (a.H / a.Hkv);
    const int64_t p = a.pos[n], r = a.row ? a.row[n] : n;
    const bool ok = p >= 0 && p < g.T && p < a.max_pages * a.P && r >= 0 && r < a.rows;
    Q *out = (Q *)a.out;
    if (!ok) {
        if (threadIdx.x == 0) {
            if (p != -1) atomicOr(a.err, SA_DEVERR_BOUNDS);
            a.lse[nh] = -INFINITY;
        }
        if (threadIdx.x < D) out[nh * D + threadIdx.x] = Q(0.f);
        return;
    }
    float qf[V];
#pragma unroll
    for (int x = 0; x < V; ++x) qf[x] = (float)((const Q *)a.q)[nh * D + sub * V + x] * a.scale2;
    const RowEdges e = row_edges(g, p);
    float m = -INFINITY, l = 0.f, acc[V];
#pragma unroll
    for (int x = 0; x < V; ++x) acc[x] = 0.f;
    for (int64_t e0 = 0; e0 < e.deg; e0 += NG) {
        const int64_t x0 = e0 + warp * G + grp;
        bool valid = x0 < e.deg;
        float kf[V], vf[V], ks = 1.f, vs = 1.f;
#pragma unroll
        for (int x = 0; x < V; ++x) kf[x] = vf[x] = 0.f;
        if (valid) {
            const int64_t j = row_edge(g, e, p, x0);
            const int64_t page = a.table[r * a.max_pages + j / a.P];
            if (page < 0 || page >= a.n_pages) {
                valid = false;
                if (sub == 0) atomicOr(a.err, SA_DEVERR_BOUNDS);
            } else {
                const int64_t at = (page * a.Hkv + kvh) * a.P + j % a.P;
                Row<T>::load(a.k, at * D + sub * V, kf);
                Row<T>::load(a.v, at * D + sub * V, vf);
                if (a.k_scale) {
                    ks = a.k_scale[at];
                    vs = a.v_scale[at];
                }
            }
        }
        float s = 0.f;
#pragma unroll
        for (int x = 0; x < V; ++x) s = fmaf(qf[x], kf[x], s);
        s = group_sum<L>(s) * ks;
        if (valid) {
            const float mn = fmaxf(m, s);
            const float base = mn == -INFINITY ? 0.f : mn;
            const float al = ex2(m - base), pe = ex2(s - base);
            l = l * al + pe;
#pragma unroll
            for (int x = 0; x < V; ++x) acc[x] = fmaf(pe * vs, vf[x], acc[x] * al);
            m = mn;
        }
    }
#pragma unroll
    for (int o = L; o < 32; o <<= 1) {
        const float mo = __shfl_xor_sync(0xffffffffu, m, o);
        const float lo = __shfl_xor_sync(0xffffffffu, l, o);
        const float mn = fmaxf(m, mo), base = mn == -INFINITY ? 0.f : mn;
        const float w0 = ex2(m - base), w1 = ex2(mo - base);
        l = l * w0 + lo * w1;
#pragma unroll
        for (int x = 0; x < V; ++x)
            acc[x] = acc[x] * w0 + __shfl_xor_sync(0xffffffffu, acc[x], o) * w1;
        m = mn;
    }
    if (grp == 0) {
#pragma unroll
        for (int x = 0; x < V; ++x) s_acc[warp][sub * V + x] = acc[x];
        if (sub == 0) {
            s_m[warp] = m;
            s_l[warp] = l;
        }
    }
    __syncthreads();
    if (threadIdx.x < D) {
        float mt = -INFINITY, lt = 0.f, o = 0.f;
        for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, s_m[w]);
        const float base = mt == -INFINITY ? 0.f : mt;
        for (int w = 0; w < kWarps; ++w) {
            const float f = ex2(s_m[w] - base);
            lt = fmaf(s_l[w], f, lt);
            o = fmaf(s_acc[w][threadIdx.x], f, o);
        }
        out[nh * D + threadIdx.x] = Q(lt == 0.f ? 0.f : o / lt);
        if (threadIdx.x == 0) a.lse[nh] = lt == 0.f ? -INFINITY : (base + lg2(lt)) * kLn2;
    }
}

template <typename T, int D>
sa_status launch_decode(const DecodeArgs &a, const GraphView &g, int64_t blocks, cudaStream_t s) {
    if (blocks > 0x7fffffffLL) return SA_ERR_UNSUPPORTED;
    SA_LAUNCH("paged_decode", s,
              paged_decode_kernel<T, D><<<(unsigned)blocks, 32 * kWarps, 0, s>>>(a, g));
    SA_CUDA_TRY(cudaGetLastError());
    return SA_OK;
}

}  // namespace

size_t sa_paged_decode_workspace(const sa_tensor *, const sa_paged_cache &, const sa_graph_s *) {
    return 0;
}

sa_status sa_paged_decode(const sa_tensor *q, const sa_paged_cache &c, const int32_t *table,
                          int64_t rows, int64_t max_pages, const int32_t *row, const int64_t *pos,
                          const sa_graph_s *g, float scale, sa_tensor *out, float *lse,
                          void *workspace, cudaStream_t s) {
    (void)workspace;
    DecodeArgs a = {};
    a.q = q->ptr;
    a.k = c.k;
    a.v = c.v;
    a.k_scale = c.k_scale;
    a.v_scale = c.v_scale;
    a.table = table;
    a.row = row;
    a.pos = pos;
    a.rows = rows;
    a.max_pages = max_pages;
    a.n_pages = c.n_pages;
    a.H = (int32_t)q->H;
    a.Hkv = (int32_t)c.Hkv;
    a.P = (int32_t)c.page_size;
    a.scale2 = scale * kLog2e;
    a.out = out->ptr;
    a.lse = lse;
    a.err = sa_device_error_word();
    if (!a.err) return SA_ERR_CUDA;
    const GraphView gv = make_view(g);
    const int64_t blocks = q->B * q->H;
#define SA_PAGED_DECODE(D)                                                            \
    switch (c.dtype) {                                                                \
        case SA_BF16: return launch_decode<__nv_bfloat16, D>(a, gv, blocks, s);       \
        case SA_FP32: return launch_decode<float, D>(a, gv, blocks, s);               \
        case SA_E4M3: return launch_decode<E4m3, D>(a, gv, blocks, s);                \
    }                                                                                 \
    break;
    switch (c.D) {
        case 32: SA_PAGED_DECODE(32)
        case 64: SA_PAGED_DECODE(64)
        case 128: SA_PAGED_DECODE(128)
    }
#undef SA_PAGED_DECODE
    return SA_ERR_UNSUPPORTED;
}
