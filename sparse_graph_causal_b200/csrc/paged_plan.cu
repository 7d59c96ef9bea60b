// paged_plan.cu -- the bookkeeping of one serving step on the GPU: block
// tables, slot maps and the free-page stack from request lengths.
//
// With L = len, n = new tokens, P = page size and a stack of c free pages:
//   cu    = exclusive prefix sum of max(n, 0)
//   back  = pages of finished requests (n = -1), prefix-summed: their places
//           on the stack, whose top is then c + sum back
//   need  = ceil((L + n) / P) - ceil(L / P), prefix-summed over the requests
//           that fit; a request is served while the inclusive sum stays
//           within the stack; its i-th new page is stack[top - 1 - (sum
//           before it) - i]
//   token t of request b: pos = L + t - cu[b], page = old table entry or new
//           page, slot = page * P + pos mod P
//
// Nothing here is worth a byte of bandwidth (20 bytes a token, 40 a request):
// the step is bound by its chain of dependent loads, barriers and launches, so
// it is one launch, a single CTA or one cluster (64 requests of one token 3.3 us a
// call in a graph, 3.7 on a stream; 2,000 requests with 60,000 tokens 11.3 and 11.5,
// with eight CTAs 15.6).  Every CTA runs the scans of
// all requests by itself and keeps what the tokens need in its shared memory;
// then the CTAs share the tokens, each found by bisection.  A cluster barrier
// orders every read of the lengths before the writes of the new ones (which
// may be the same array) and returned pages before taken ones.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "paged_common.cuh"
#include "sa_internal.cuh"

namespace {

namespace cg = cooperative_groups;

constexpr unsigned kFull = 0xffffffffu;
constexpr int kRun = 4;  // tokens of a thread at a time

// Sums that stop at the largest value (they are compared with stack sizes).
__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) {
    const uint32_t s = a + b;
    return s < a ? 0xffffffffu : s;
}

// Inclusive prefix sums over the block of a 64-bit and a 32-bit value per
// thread, with their totals; one barrier.  Returns whether any `flag` is set.
template <int NW, typename A>
__device__ __forceinline__ bool block_scan(A &x, uint32_t &y, A &x_all, uint32_t &y_all, bool flag,
                                           A *s_x, uint32_t *s_y) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const A u = __shfl_up_sync(kFull, x, o);
        const uint32_t v = __shfl_up_sync(kFull, y, o);
        if (lane >= o) x += u, y = add_sat(y, v);
    }
    if (lane == 31) s_x[warp] = x, s_y[warp] = y;
    const bool any = __syncthreads_or(flag);
    A u = lane < NW ? s_x[lane] : 0;
    uint32_t v = lane < NW ? s_y[lane] : 0;
#pragma unroll
    for (int o = 1; o < NW; o <<= 1) {
        const A p = __shfl_up_sync(kFull, u, o);
        const uint32_t q = __shfl_up_sync(kFull, v, o);
        if (lane >= o) u += p, v = add_sat(v, q);
    }
    x_all = __shfl_sync(kFull, u, NW - 1);
    y_all = __shfl_sync(kFull, v, NW - 1);
    const A before = __shfl_sync(kFull, u, warp ? warp - 1 : 0);
    const uint32_t before_y = __shfl_sync(kFull, v, warp ? warp - 1 : 0);
    if (warp) x += before, y = add_sat(y, before_y);
    return any;
}

struct PlanArgs {
    sa_paged_step s;
    Divide page;
    int32_t size;  // power of two above B
};

// First new page of a request counted from the top of the stack (a finished
// one: where its pages go on the stack), or kRefused: it is not served.
constexpr int kRefused = -1;

// NT threads; PER requests each (consecutive ones), kept in registers.
template <int NT, int PER>
__global__ void __launch_bounds__(NT) paged_plan_kernel(const PlanArgs args) {
    chain_begin();
    const sa_paged_step &a = args.s;
    constexpr int NW = NT / 32;
    extern __shared__ int32_t smem[];
    __shared__ int64_t s_x[NW];
    __shared__ uint32_t s_y[NW], s_z[NW], s_w[NW], s_taken;
    const int B = (int)a.B, tid = threadIdx.x;
    // the end of each request's tokens (clipped to capacity), its length (-1 -
    // length if it is finished) and its first new page
    // (s_end: a power of two above B of entries, the rest never reached)
    const int a_size = args.size;
    int32_t *s_end = smem, *s_len = smem + a_size, *s_new = s_len + B;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ncta = (int)cluster.num_blocks();
    const int64_t room = a.max_pages * a.page_size;
    const uint32_t P = args.page.by;
    const int b0 = tid * PER;
    // ceil(x / P) for 0 <= x <= room < 2^31
    auto pages = [&](int64_t x) { return x ? divide((uint32_t)x - 1, args.page) + 1 : 0; };

    int64_t len[PER];
    int32_t nn[PER];
    const int64_t count = *a.free_count;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        len[k] = b0 + k < B ? a.len[b0 + k] : 0;
        nn[k] = b0 + k < B ? a.n_new[b0 + k] : 0;
    }
    int64_t tokens = 0, tokens_all;
    uint32_t back = 0, back_all, used[PER];
    bool sane[PER], finished = false;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        tokens += nn[k] > 0 ? nn[k] : 0;
        sane[k] = len[k] >= 0 && len[k] <= room;
        used[k] = sane[k] ? pages(len[k]) : 0;
        if (nn[k] == -1) {
            back = add_sat(back, used[k]);
            finished = true;
        }
    }
    if (tid == 0) s_taken = 0;
    for (int b = B + tid; b < a_size; b += NT) s_end[b] = 0x7fffffff;
    int64_t cu = tokens;
    uint32_t bk = back;
    finished = block_scan<NW>(cu, bk, tokens_all, back_all, finished, s_x, s_y);
    const bool stack_ok = count >= 0 && count <= a.n_stack;
    const uint32_t space = stack_ok ? (uint32_t)(a.n_stack - count) : 0;  // places left
    cu -= tokens;
    // (a saturated sum is above every space, and so are the sums before it here)
    bk = bk == 0xffffffffu ? bk : bk - back;

    // which requests fit, whose pages come back, and what is needed
    uint32_t need = 0, kept = 0, want[PER];
    int32_t state[PER];
    {
        int64_t c = cu;
        uint32_t b = bk;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            want[k] = 0;
            state[k] = SA_PAGED_REFUSED;
            if (b0 + k >= B) continue;
            const int64_t n = nn[k] > 0 ? nn[k] : 0;
            c += n;
            if (nn[k] == -1) {
                b = add_sat(b, used[k]);
                if (sane[k] && stack_ok && (b <= space || used[k] == 0)) {
                    state[k] = SA_PAGED_OK;
                    kept += used[k];
                }
            } else if (nn[k] >= 0 && sane[k] && len[k] + n <= room && c <= a.capacity) {
                state[k] = SA_PAGED_NO_PAGES;  // until its pages are known to be there
                want[k] = pages(len[k] + n) - used[k];
                need += want[k];
            }
        }
    }
    uint32_t need_upto = need, kept_upto = kept, need_all, kept_all;
    block_scan<NW>(need_upto, kept_upto, need_all, kept_all, false, s_z, s_w);
    const uint32_t top = stack_ok ? (uint32_t)count + kept_all : 0;
    uint32_t upto = need_upto - need, place = (uint32_t)count + kept_upto - kept, taken = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int b = b0 + k;
        if (b >= B) continue;
        int32_t first = kRefused;
        if (nn[k] == -1) {
            if (state[k] == SA_PAGED_OK) {
                first = (int32_t)place;
                place += used[k];
            }
        } else if (state[k] == SA_PAGED_NO_PAGES) {
            upto += want[k];
            if (want[k] == 0 || upto <= top) {
                state[k] = SA_PAGED_OK;
                first = want[k] ? (int32_t)(upto - want[k]) : 0;
                if (want[k]) taken = upto;  // (sums only grow: the last is the largest)
            }
        }
        cu += nn[k] > 0 ? nn[k] : 0;
        if (rank == 0) a.cu_new[b + 1] = cu;
        s_end[b] = (int32_t)(cu < a.capacity ? cu : a.capacity);
        s_len[b] = !sane[k] ? 0 : nn[k] == -1 ? -1 - (int32_t)len[k] : (int32_t)len[k];
        s_new[b] = first;
    }
    if (taken) atomicMax(&s_taken, taken);
    if (rank == 0 && tid == 0) a.cu_new[0] = 0;
    __syncthreads();

    // returned pages go on the stack: a warp per finished request
    if (finished) {
        const int warp = rank * NW + (tid >> 5), lane = tid & 31;
        for (int b = warp; b < B; b += ncta * NW) {
            if (s_len[b] >= 0 || s_new[b] == kRefused) continue;
            const int32_t n = (int32_t)pages(-1 - s_len[b]);
            const int32_t *from = a.block_table + (int64_t)b * a.max_pages;
            int32_t *to = a.free_pages + s_new[b];
            for (int32_t p = lane; p < n; p += 128) {
                int32_t x[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) x[y] = p + 32 * y < n ? from[p + 32 * y] : 0;
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    if (p + 32 * y < n) to[p + 32 * y] = x[y];
            }
        }
    }
    if (ncta > 1) cluster.sync();
    else if (finished) __syncthreads();

    // new state (every CTA has read the old one)
    if (rank == 0) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int b = b0 + k;
            if (b >= B) continue;
            a.status[b] = state[k];
            a.len_out[b] = state[k] != SA_PAGED_OK ? len[k] : nn[k] == -1 ? 0 : len[k] + nn[k];
        }
        if (tid == 0) *a.free_count_out = stack_ok ? (int64_t)(top - s_taken) : count;
    }

    // tokens: kRun of a thread, NT apart, so that their loads overlap and
    // neighbours store together
    const int32_t capacity = (int32_t)a.capacity;
    for (int32_t t0 = rank * NT * kRun; t0 < capacity; t0 += ncta * NT * kRun) {
        int32_t page[kRun], row[kRun], pos[kRun];
        uint32_t off[kRun];
        int32_t *entry[kRun];
        // requests whose tokens end before the token (without branches: four
        // searches side by side)
        int32_t lo[kRun] = {};
        for (int n = a_size >> 1; n; n >>= 1)
#pragma unroll
            for (int x = 0; x < kRun; ++x)
                lo[x] += s_end[lo[x] + n - 1] <= t0 + x * NT + tid ? n : 0;
#pragma unroll
        for (int x = 0; x < kRun; ++x) {
            const int32_t t = t0 + x * NT + tid;
            const int b = lo[x];
            row[x] = pos[x] = page[x] = -1;
            off[x] = 0;
            entry[x] = nullptr;
            if (t < capacity && b < B && s_new[b] != kRefused) {
                const int32_t L = s_len[b];
                row[x] = b;
                pos[x] = L + (int32_t)(t - (b ? s_end[b - 1] : 0));
                const uint32_t p = divide((uint32_t)pos[x], args.page), u = pages(L);
                off[x] = (uint32_t)pos[x] - p * P;
                int32_t *e = a.block_table + (int64_t)b * a.max_pages + p;
                if (p < u) {
                    page[x] = *e;
                } else {
                    page[x] = __ldcg(a.free_pages + (top - 1 - ((uint32_t)s_new[b] + (p - u))));
                    if (off[x] == 0) entry[x] = e;
                }
            }
        }
#pragma unroll
        for (int x = 0; x < kRun; ++x) {
            const int32_t t = t0 + x * NT + tid;
            if (t >= capacity) continue;
            if (entry[x]) *entry[x] = page[x];
            a.slot[t] = page[x] >= 0 ? (int64_t)page[x] * P + off[x] : -1;
            a.pos[t] = pos[x];
            a.row[t] = row[x];
        }
    }
}

// Whether the device takes clusters of 16 of this kernel (beyond the portable
// eight), asked once per kernel and device.
template <int NT, int PER>
bool takes_sixteen(size_t smem) {
    static std::atomic<int8_t> known[64];  // 0: not asked, 1: no, 2: yes
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    int8_t k = known[dev].load(std::memory_order_relaxed);
    if (k == 0) {
        const auto fn = paged_plan_kernel<NT, PER>;
        int clusters = 0;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        cfg.gridDim = dim3(16);
        cfg.blockDim = dim3(NT);
        cfg.dynamicSmemBytes = smem;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 16;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const bool ok =
            cudaFuncSetAttribute((const void *)fn, cudaFuncAttributeNonPortableClusterSizeAllowed,
                                 1) == cudaSuccess &&
            cudaOccupancyMaxActiveClusters(&clusters, fn, &cfg) == cudaSuccess && clusters > 0;
        if (!ok) cudaGetLastError();  // an answer, not a failure
        k = ok ? 2 : 1;
        known[dev].store(k, std::memory_order_relaxed);
    }
    return k == 2;
}

template <int NT, int PER>
sa_status launch_plan(const PlanArgs &p, cudaStream_t s) {
    const void *fn = (const void *)paged_plan_kernel<NT, PER>;
    // the opt-in holds for the largest B of this variant
    SA_CUDA_TRY(sa_smem_optin(fn, 4 * 4 * PER * NT));
    // as many CTAs as give each one turn of tokens
    int ncta = p.s.capacity > 2048 ? 8 : 1;
    if (p.s.capacity > 8 * NT * kRun && takes_sixteen<NT, PER>(4 * 4 * PER * NT)) ncta = 16;
    cudaError_t e = cudaSuccess;
    SA_LAUNCH("paged_plan", s,
              e = launch_chained(paged_plan_kernel<NT, PER>, dim3(ncta), NT,
                                 4 * (size_t)(p.size + 2 * p.s.B), s, ncta, p));
    SA_CUDA_TRY(e);
    return SA_OK;
}

}  // namespace

sa_status sa_paged_plan(const sa_paged_step &step, cudaStream_t s) {
    PlanArgs p = {step, make_divide((uint32_t)step.page_size), 1};
    while (p.size <= step.B) p.size *= 2;
    static_assert(SA_PAGED_MAX_REQUESTS <= 8 * 1024, "requests per thread");
    if (p.s.B <= 256 && p.s.capacity <= 2048) return launch_plan<256, 1>(p, s);
    if (p.s.B <= 1024) return launch_plan<1024, 1>(p, s);
    if (p.s.B <= 2048) return launch_plan<1024, 2>(p, s);
    return p.s.B <= 4096 ? launch_plan<1024, 4>(p, s) : launch_plan<1024, 8>(p, s);
}
