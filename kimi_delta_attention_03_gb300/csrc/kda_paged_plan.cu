// kda_paged_plan.cu — block tables, token positions and cache slots from the requests' lengths.
//
// Per request n: cached c_n tokens, a run of r_n new ones, held_n pages in its table.
//     need_n  = max(ceil((c_n + r_n) / page) - held_n, 0)
//     cum_n   = need_0 + ... + need_n                     (inclusive)
//     given_n = need_n == 0 or cum_n <= avail             (cum never falls: a prefix is served)
// avail counts the free list after the released requests' pages are pushed on its end, in request
// order; new page j of request n is the free list's entry avail - 1 - (cum_n - need_n) - j.
//
// What bounds it: latency.  The bytes (28 per request, 8 per token, 8 per page) take a microsecond
// at HBM rate even for 64K tokens; the chain launch -> lengths -> scan -> page -> slot does not
// shrink with size.  So one launch does it all: every CTA of one cluster scans all requests itself
// (two 64-bit sums per request, shuffles and one barrier) instead of waiting for another's scan,
// and takes its share of the tokens.  Only released pages cross CTAs; a cluster barrier orders
// those, and a call that releases nothing skips it.
#include <cooperative_groups.h>

#include <algorithm>

#include "kda_common.cuh"
#include "kda_paged.cuh"

namespace kda {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanCluster = 8;

// One request as every CTA of the cluster sees it.
struct PlanSeq {
    int32_t cached;  // -1: not served
    int32_t held;    // pages it keeps
    int32_t need;    // new pages; minus the number of pages it gives back
    int32_t excl;    // new pages asked for (or pages given back) by those before it
};

__device__ __forceinline__ int64_t warp_scan(int64_t x, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(~0u, x, d);
        if (lane >= d) x += y;
    }
    return x;
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PlanArgs a, int* status) {
    namespace cg = cooperative_groups;
    extern __shared__ __align__(16) unsigned char smem[];
    PlanSeq* seq = reinterpret_cast<PlanSeq*>(smem);
    int32_t* cu = reinterpret_cast<int32_t*>(seq + a.num_seqs);
    __shared__ int64_t warp_need[kPlanThreads / 32], warp_back[kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x, ctas = gridDim.x;  // the grid is one cluster
    const int N = a.num_seqs, per = (N + kPlanThreads - 1) / kPlanThreads;
    const int n0 = min(tid * per, N), n1 = min(n0 + per, N);
    bool bad = false;

    // 1. lengths, needs and released pages of this thread's requests
    int64_t need = 0, back = 0;
    for (int n = n0; n < n1; ++n) {
        const int c0 = a.cu[n], c1 = a.cu[n + 1], held = a.held[n];
        const int cached = a.cached[n];
        const bool gone = a.release && a.release[n] != 0;
        const int64_t total = ((int64_t)cached + c1 - c0 + a.page_size - 1) / a.page_size;
        const bool sane = c0 >= 0 && c1 >= c0 && c1 <= a.total_tokens && held >= 0 &&
                          held <= a.width && cached >= 0 &&
                          (gone || cached <= (int64_t)held * a.page_size);
        bad |= !sane;
        const bool takes = sane && !gone && total <= a.width;
        PlanSeq s;
        s.cached = takes ? cached : -1;
        s.held = sane ? held : 0;
        s.need = takes && total > held ? (int32_t)(total - held) : 0;
        s.excl = 0;
        seq[n] = s;
        cu[n] = c0;
        if (n == N - 1) cu[N] = c1;
        need += s.need;
        if (gone) back += s.held;
    }
    // 2. exclusive prefix sums over the requests
    const int64_t need_in = warp_scan(need, lane), back_in = warp_scan(back, lane);
    if (lane == 31) {
        warp_need[warp] = need_in;
        warp_back[warp] = back_in;
    }
    __syncthreads();
    int64_t need_at = need_in - need, back_at = back_in - back, back_all = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) {
            need_at += warp_need[w];
            back_at += warp_back[w];
        }
        back_all += warp_back[w];
    }
    int64_t count = *a.free_count;
    bad |= count < 0 || count + back_all > a.capacity;
    count = min(max(count, (int64_t)0), (int64_t)a.capacity);
    const int64_t avail = min(count + back_all, (int64_t)a.capacity);

    // 3. who is served; the requests' own results
    int64_t used = 0;  // new pages of this thread's served requests
    for (int n = n0; n < n1; ++n) {
        PlanSeq s = seq[n];
        const bool gone = a.release && a.release[n] != 0;
        const int64_t excl = need_at;
        need_at += s.need;
        const bool given = s.cached >= 0 && (s.need == 0 || need_at <= avail);
        const int cached = gone ? 0 : max(a.cached[n], 0);
        if (gone) {  // its pages go to the list's entries count + excl ...
            s.need = -s.held;
            s.excl = (int32_t)min(back_at, (int64_t)INT32_MAX);
            back_at += s.held;
            s.held = 0;
        } else {
            if (!given) s.need = 0;
            s.excl = (int32_t)min(excl, (int64_t)INT32_MAX);
            used += s.need;
        }
        s.cached = given ? cached : -1 - cached;
        seq[n] = s;
        if (n % ctas == rank) {
            a.context[n] = given ? cached + cu[n + 1] - cu[n] : cached;
            a.held_out[n] = gone ? 0 : s.held + s.need;
        }
    }
    used = warp_scan(used, lane);
    __syncthreads();  // the warps' sums are read and the requests written
    if (lane == 31) warp_need[warp] = used;
    const int warps = ctas * (kPlanThreads / 32), first = rank * (kPlanThreads / 32) + warp;
    if (back_all > 0) {  // released pages, a warp per request; other CTAs may take them
        for (int n = first; n < N; n += warps) {
            const PlanSeq s = seq[n];
            const int64_t at = count + s.excl;
            for (int j = lane; j < -s.need; j += 32)
                if (at + j < a.capacity) a.free_list[at + j] = a.tables[(int64_t)n * a.width + j];
        }
        cg::this_cluster().sync();
    } else {
        __syncthreads();
    }
    if (rank == 0 && tid == 0) {
        int64_t sum = 0;
        for (int w = 0; w < kPlanThreads / 32; ++w) sum += warp_need[w];
        *a.free_out = (int32_t)(avail - sum);
    }

    // 4. new table entries: a warp per request
    for (int n = first; n < N; n += warps) {
        const PlanSeq s = seq[n];
        for (int j = lane; j < s.need; j += 32)
            a.tables[(int64_t)n * a.width + s.held + j] = a.free_list[avail - 1 - s.excl - j];
    }
    // 5. positions and slots: a thread per token.  A page taken in this call is read from the free
    // list itself, so nothing here waits for step 4.
    const int64_t rows = min((int64_t)max(cu[N], 0), a.total_tokens);
    for (int64_t t = (int64_t)rank * kPlanThreads + tid; t < a.total_tokens;
         t += (int64_t)ctas * kPlanThreads) {
        int pos = 0, slot = -1;
        if (t < rows && t >= cu[0]) {
            const int n = seq_of_row(cu, N, (int)t);
            const PlanSeq s = seq[n];
            pos = (s.cached >= 0 ? s.cached : -1 - s.cached) + (int)t - cu[n];
            const int b = pos / a.page_size;
            if (s.cached >= 0 && b < s.held + s.need) {
                const int page = b < s.held ? a.tables[(int64_t)n * a.width + b]
                                            : a.free_list[avail - 1 - s.excl - (b - s.held)];
                slot = (int)((unsigned)page * (unsigned)a.page_size) + pos % a.page_size;
            }
        }
        a.positions[t] = pos;
        a.slots[t] = slot;
    }
    if (bad) report_status(status, KDA_ERR_INVALID_ARG);
}

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs& a, int* status, cudaStream_t stream) {
    const size_t smem = (size_t)a.num_seqs * sizeof(PlanSeq) + ((size_t)a.num_seqs + 1) * 4;
    cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    // one CTA up to 4 tokens a thread, then a cluster
    const int ctas = a.total_tokens <= 4 * kPlanThreads ? 1 : kPlanCluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_plan_kernel, a, status);
}

}  // namespace kda
