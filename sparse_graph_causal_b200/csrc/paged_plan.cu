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
// the step is bound by its chain of dependent loads and by launches, so it is
// one launch, a single CTA or one cluster.  Every CTA runs the scans of all
// requests by itself (three 64-bit sums over 1,024 threads) and keeps what
// the tokens need in its shared memory; then the CTAs share the tokens.  A
// cluster barrier orders every read of the lengths before the writes of the
// new ones (which may be the same array) and returned pages before taken ones.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sa_internal.cuh"

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

// Inclusive prefix sum of one value per thread over the block.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t *s_part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // the last use of s_part is over
    if (lane == 31) s_part[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int64_t p = s_part[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, p, o);
            if (lane >= o) p += y;
        }
        s_part[lane] = p;
    }
    __syncthreads();
    return x + (warp ? s_part[warp - 1] : 0);
}

// What the tokens of request b need, in shared memory: the end of its tokens
// (clipped to capacity), its length, and its first new page counted from the
// top of the stack (kRefused: it is not served).
constexpr int kRefused = -1;

// MAXPER: requests per thread (consecutive ones), kept in registers.
template <int MAXPER>
__global__ void __launch_bounds__(kThreads) paged_plan_kernel(sa_paged_step a) {
    static_assert(kWarps == 32, "one warp scans the warps' sums");
    extern __shared__ int32_t smem[];
    __shared__ int64_t s_part[kWarps];
    __shared__ int64_t s_free;
    const int B = (int)a.B, tid = threadIdx.x;
    int32_t *s_end = smem, *s_len = smem + B, *s_new = smem + 2 * B;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ncta = (int)cluster.num_blocks();
    const int64_t P = a.page_size, room = a.max_pages * P;
    const int per = (B + kThreads - 1) / kThreads, b0 = tid * per;

    int64_t len[MAXPER];
    int32_t nn[MAXPER];
    if (tid == 0) s_free = *a.free_count;
    int64_t tokens = 0, back = 0;
#pragma unroll
    for (int k = 0; k < MAXPER; ++k) {
        const int b = b0 + k;
        const bool in = k < per && b < B;
        len[k] = in ? a.len[b] : 0;
        nn[k] = in ? a.n_new[b] : 0;
    }
#pragma unroll
    for (int k = 0; k < MAXPER; ++k) {
        tokens += nn[k] > 0 ? nn[k] : 0;
        const bool sane = len[k] >= 0 && len[k] <= room;
        back += nn[k] == -1 && sane ? (len[k] + P - 1) / P : 0;
    }
    const int64_t tokens_upto = block_scan(tokens, s_part);
    const int64_t back_upto = block_scan(back, s_part);
    const int64_t count = s_free;
    const bool stack_ok = count >= 0 && count <= a.n_stack;
    const int64_t space = stack_ok ? a.n_stack - count : -1;  // places left on the stack

    // which requests fit, whose pages come back, and what is needed
    int64_t cu = tokens_upto - tokens, bk = back_upto - back, need = 0, kept = 0;
    int64_t want[MAXPER];
    int32_t state[MAXPER];
#pragma unroll
    for (int k = 0; k < MAXPER; ++k) {
        const int b = b0 + k;
        want[k] = 0;
        state[k] = SA_PAGED_REFUSED;
        if (!(k < per && b < B)) continue;
        const bool sane = len[k] >= 0 && len[k] <= room;
        const int64_t used = sane ? (len[k] + P - 1) / P : 0, n = nn[k] > 0 ? nn[k] : 0;
        cu += n;
        if (rank == 0) a.cu_new[b + 1] = cu;
        s_end[b] = (int32_t)(cu < a.capacity ? cu : a.capacity);
        s_len[b] = sane ? (int32_t)len[k] : 0;
        s_new[b] = kRefused;
        if (nn[k] == -1) {
            bk += used;
            if (sane && (bk <= space || (used == 0 && stack_ok))) {
                state[k] = SA_PAGED_OK;
                kept += used;
            }
        } else if (nn[k] >= 0 && sane && len[k] + n <= room && cu <= a.capacity) {
            state[k] = SA_PAGED_NO_PAGES;  // until its pages are known to be there
            want[k] = (len[k] + n + P - 1) / P - used;
            need += want[k];
        }
    }
    const int64_t need_upto = block_scan(need, s_part);
    const int64_t kept_upto = block_scan(kept, s_part);
    __syncthreads();
    const int64_t kept_all = s_part[kWarps - 1];
    const int64_t top = stack_ok ? count + kept_all : 0;
    int64_t upto = need_upto - need, place = count + kept_upto - kept, taken = 0;
#pragma unroll
    for (int k = 0; k < MAXPER; ++k) {
        const int b = b0 + k;
        if (!(k < per && b < B)) continue;
        const int64_t used = (int64_t)(s_len[b] + P - 1) / P;
        if (nn[k] == -1) {
            // (s_new of a finished request: where its pages go on the stack)
            if (state[k] == SA_PAGED_OK) {
                s_new[b] = (int32_t)place;
                place += used;
            }
        } else if (state[k] == SA_PAGED_NO_PAGES) {
            upto += want[k];
            if (want[k] == 0 || upto <= top) {
                state[k] = SA_PAGED_OK;
                s_new[b] = want[k] ? (int32_t)(upto - want[k]) : 0;
                taken += want[k];
            }
        }
    }
    const int64_t taken_upto = block_scan(taken, s_part);  // also: shared arrays are complete
    if (rank == 0 && tid == 0) a.cu_new[0] = 0;

    // returned pages go on the stack: a warp per finished request
    const int warp = rank * kWarps + (tid >> 5), nwarp = ncta * kWarps, lane = tid & 31;
    for (int b = warp; b < B; b += nwarp) {
        if (a.n_new[b] != -1 || s_new[b] == kRefused) continue;
        const int64_t used = (int64_t)(s_len[b] + P - 1) / P;
        for (int64_t p = lane; p < used; p += 32)
            a.free_pages[s_new[b] + p] = a.block_table[(int64_t)b * a.max_pages + p];
    }
    cluster.sync();

    // new state (every CTA has read the old one)
#pragma unroll
    for (int k = 0; k < MAXPER; ++k) {
        const int b = b0 + k;
        if (rank != 0 || !(k < per && b < B)) continue;
        a.status[b] = state[k];
        a.len_out[b] = state[k] != SA_PAGED_OK ? len[k]
                       : nn[k] == -1           ? 0
                                               : len[k] + nn[k];
    }
    if (rank == 0 && tid == kThreads - 1) *a.free_count_out = stack_ok ? top - taken_upto : count;

    // tokens: a run of kRun consecutive ones per thread, the request of the
    // first found by bisection
    constexpr int kRun = 4;
    const int64_t step = (int64_t)ncta * kThreads * kRun;
    for (int64_t t0 = ((int64_t)rank * kThreads + tid) * kRun; t0 < a.capacity; t0 += step) {
        int lo = 0, hi = B;  // first request whose tokens end after t0
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s_end[mid] > t0) hi = mid;
            else lo = mid + 1;
        }
        int b = lo;
#pragma unroll
        for (int x = 0; x < kRun; ++x) {
            const int64_t t = t0 + x;
            if (t >= a.capacity) break;
            while (b < B && s_end[b] <= t) ++b;
            int64_t slot = -1, pos = -1;
            int32_t row = -1;
            if (b < B && s_new[b] != kRefused) {
                const int32_t L = s_len[b];
                const int64_t first = b ? s_end[b - 1] : 0;
                const int64_t used = ((int64_t)L + P - 1) / P;
                pos = L + (t - first);
                row = b;
                const int64_t p = pos / P, off = pos - p * P;
                int32_t *entry = a.block_table + (int64_t)b * a.max_pages + p;
                int32_t page;
                if (p < used) {
                    page = *entry;
                } else {
                    page = __ldcg(a.free_pages + (top - 1 - (s_new[b] + (p - used))));
                    if (off == 0) *entry = page;
                }
                slot = page >= 0 ? (int64_t)page * P + off : -1;
            }
            a.slot[t] = slot;
            a.pos[t] = pos;
            a.row[t] = row;
        }
    }
}

template <int MAXPER>
sa_status launch_plan(const sa_paged_step &p, cudaStream_t s) {
    const void *fn = (const void *)paged_plan_kernel<MAXPER>;
    const int smem = 3 * 4 * (int)p.B;
    // the opt-in holds for the largest B of this variant
    const int most = 3 * 4 * MAXPER * kThreads;
    SA_CUDA_TRY(sa_smem_optin(fn, most));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    const int ncta = p.capacity > 2 * kThreads ? 8 : 1;
    cfg.gridDim = dim3(ncta);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ncta;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaSuccess;
    SA_LAUNCH("paged_plan", s, e = cudaLaunchKernelEx(&cfg, paged_plan_kernel<MAXPER>, p));
    SA_CUDA_TRY(e);
    return SA_OK;
}

}  // namespace

sa_status sa_paged_plan(const sa_paged_step &p, cudaStream_t s) {
    static_assert(SA_PAGED_MAX_REQUESTS <= 8 * kThreads, "requests per thread");
    return p.B <= kThreads ? launch_plan<1>(p, s) : launch_plan<8>(p, s);
}
