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
// shrink with size: 64 requests of 4 tokens take 5.0 us, 512 requests of up to 512 tokens 8.3 us.
// So one launch does it all, and no block waits for another: each scans all requests itself (two
// 64-bit sums per request, shuffles and one barrier) and takes its share of the tokens.  A page
// released in this call is looked up in its old table row instead of the list entry that another
// block is writing.
#include <algorithm>

#include "kda_common.cuh"
#include "kda_paged.cuh"

namespace kda {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanTokens = 4;  // consecutive tokens of a thread

// One request as every block sees it.
struct PlanSeq {
    int32_t cached;  // -1 - cached: not served
    int32_t held;    // pages it keeps
    int32_t need;    // new pages; minus the number of pages it gives back
    int32_t excl;    // new pages asked for by those before it
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
    extern __shared__ __align__(16) unsigned char smem[];
    const int N = a.num_seqs;
    PlanSeq* seq = reinterpret_cast<PlanSeq*>(smem);
    int32_t* cu = reinterpret_cast<int32_t*>(seq + N);  // [N + 1]
    int32_t* given_back = cu + N + 1;                   // [N + 1]: pages released before request n
    __shared__ int64_t warp_need[kPlanThreads / 32], warp_back[kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x, ctas = gridDim.x;
    const int per = (N + kPlanThreads - 1) / kPlanThreads;
    const int n0 = min(tid * per, N), n1 = min(n0 + per, N);
    bool bad = false;

    // 1. lengths, needs and released pages of this thread's requests
    int64_t count = *a.free_count;
    int64_t need = 0, back = 0;
    for (int n = n0; n < n1; ++n) {
        const int c0 = a.cu[n], c1 = a.cu[n + 1], held = a.held[n], cached = a.cached[n];
        const bool gone = a.release && a.release[n] != 0;
        const int64_t total = ((int64_t)cached + c1 - c0 + a.page_size - 1) / a.page_size;
        const bool sane = c0 >= 0 && c1 >= c0 && c1 <= a.total_tokens && held >= 0 &&
                          held <= a.width && cached >= 0 &&
                          (gone || cached <= (int64_t)held * a.page_size);
        bad |= !sane;
        const bool takes = sane && !gone && total <= a.width;
        PlanSeq s;
        s.cached = gone ? -1 : takes ? cached : -1 - max(cached, 0);
        s.held = gone || !sane ? 0 : held;
        s.need = gone ? (sane ? -held : 0) : takes && total > held ? (int32_t)(total - held) : 0;
        s.excl = 0;
        seq[n] = s;
        cu[n] = c0;
        if (n == N - 1) cu[N] = c1;
        if (s.need > 0) need += s.need;
        else back -= s.need;
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
    bad |= count < 0 || count + back_all > a.capacity;
    count = min(max(count, (int64_t)0), (int64_t)a.capacity);
    const int64_t avail = min(count + back_all, (int64_t)a.capacity);

    // 3. who is served; the requests' own results
    int64_t used = 0;  // new pages of this thread's served requests
    for (int n = n0; n < n1; ++n) {
        PlanSeq s = seq[n];
        given_back[n] = (int32_t)min(back_at, (int64_t)INT32_MAX);
        s.excl = (int32_t)min(need_at, (int64_t)INT32_MAX);
        if (s.need > 0) {
            need_at += s.need;
            if (need_at > avail) {
                s.need = 0;
                s.cached = -1 - s.cached;
            }
            used += s.need;
        } else {
            back_at -= s.need;
        }
        seq[n] = s;
        if (n % ctas == rank) {
            a.context[n] = s.cached >= 0 ? s.cached + cu[n + 1] - cu[n] : -1 - s.cached;
            a.held_out[n] = s.held + max(s.need, 0);
        }
    }
    if (n1 == N && n0 < N) given_back[N] = (int32_t)min(back_all, (int64_t)INT32_MAX);
    used = warp_scan(used, lane);
    __syncthreads();  // the warps' sums are read and the requests written
    if (lane == 31) warp_need[warp] = used;
    __syncthreads();
    if (rank == 0 && tid == 0) {
        int64_t sum = 0;
        for (int w = 0; w < kPlanThreads / 32; ++w) sum += warp_need[w];
        *a.free_out = (int32_t)(avail - sum);
    }

    // Entry i < avail of the list with the released pages on its end.
    auto listed = [&](int64_t i) {
        if (i < count) return a.free_list[i];
        const int j = (int)(i - count);
        const int n = seq_of_row(given_back, N, j);
        return a.tables[(int64_t)n * a.width + j - given_back[n]];
    };
    // 4. released pages onto the list and new table entries: a warp per request
    const int warps = ctas * (kPlanThreads / 32);
    for (int n = rank * (kPlanThreads / 32) + warp; n < N; n += warps) {
        const PlanSeq s = seq[n];
        int32_t* row = a.tables + (int64_t)n * a.width;
        for (int j = lane; j < s.need; j += 32) row[s.held + j] = listed(avail - 1 - s.excl - j);
        const int64_t at = count + given_back[n];
        for (int j = lane; j < -s.need; j += 32)
            if (at + j < a.capacity) a.free_list[at + j] = row[j];
    }
    // 5. positions and slots of four consecutive tokens a thread.  A page taken in this call comes
    // from the list, so nothing here waits for step 4.
    const int64_t rows = min((int64_t)max(cu[N], 0), a.total_tokens);
    for (int64_t t0 = ((int64_t)rank * kPlanThreads + tid) * kPlanTokens; t0 < a.total_tokens;
         t0 += (int64_t)ctas * kPlanThreads * kPlanTokens) {
        int pos[kPlanTokens], slot[kPlanTokens];
        int n = -1, end = 0, last = -1, page = 0;
        PlanSeq s = {};
#pragma unroll
        for (int i = 0; i < kPlanTokens; ++i) {
            const int64_t t = t0 + i;
            pos[i] = 0;
            slot[i] = -1;
            if (t >= rows || t < cu[0]) continue;
            if (n < 0 || t >= end) {
                n = seq_of_row(cu, N, (int)t);
                end = cu[n + 1];
                s = seq[n];
                last = -1;
            }
            pos[i] = (s.cached >= 0 ? s.cached : -1 - s.cached) + (int)t - cu[n];
            const int b = pos[i] / a.page_size;
            if (s.cached >= 0 && b < s.held + s.need) {
                if (b != last) {
                    page = b < s.held ? a.tables[(int64_t)n * a.width + b]
                                      : listed(avail - 1 - s.excl - (b - s.held));
                    last = b;
                }
                slot[i] = (int)((unsigned)page * (unsigned)a.page_size) + pos[i] % a.page_size;
            }
        }
#pragma unroll
        for (int i = 0; i < kPlanTokens; ++i)
            if (t0 + i < a.total_tokens) {
                a.positions[t0 + i] = pos[i];
                a.slots[t0 + i] = slot[i];
            }
    }
    if (bad) report_status(status, KDA_ERR_INVALID_ARG);
}

constexpr size_t plan_smem(int num_seqs) { return (size_t)num_seqs * (sizeof(PlanSeq) + 8) + 8; }

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs& a, int* status, cudaStream_t stream) {
    static std::atomic<uint64_t> raised{0};
    const size_t smem = plan_smem(a.num_seqs);
    if (smem > 40 * 1024) {
        const cudaError_t e = raise_smem(paged_plan_kernel, plan_smem(kPlanMaxSeqs), raised);
        if (e != cudaSuccess) return e;
    }
    const int64_t per = kPlanThreads * kPlanTokens;
    const int ctas = (int)std::min<int64_t>(std::max<int64_t>((a.total_tokens + per - 1) / per, 1), kPlanSMs);
    paged_plan_kernel<<<ctas, kPlanThreads, smem, stream>>>(a, status);
    return cudaGetLastError();
}

}  // namespace kda
