// kda_verify.cu — verification of drafted tokens against the target's probabilities.
//
// A run of L tokens holds what came before and L - 1 drafts; row i of the run judges draft x_i =
// token i + 1 from given random numbers u_i in [0, 1) and e_v ~ Exp(1):
//     it holds if u_i q_i(x_i) < p_i(x_i)            (probability min(1, p / q))
//     a = the first row whose draft does not hold, or L - 1
//     w = max(p_a - q_a, 0) where a draft fell (p_a itself if that is zero everywhere), else p_a
//     next token = argmax_v w_v / e_v, ties to the lowest v
// The race w / e picks v with probability w_v / sum w: it needs no sum over the vocabulary, so its
// result does not depend on an order of summation, and one pass over three rows decides.
// Certain drafts (no q): q_i is 1 at x_i and 0 elsewhere.
//
// What bounds it: one row each of p, q and e per request, read once; the accept tests touch single
// entries.  64 requests of 131,072 fp32 entries (92.3 MB) take 18.4 us, 75% of the measured copy
// bandwidth: 512 CTAs are one wave of three or four to an SM.  A single request of 32,000 takes 4.5
// us, launch and latency.  A cluster of 8 CTAs shares a request's vocabulary, so that few requests
// still use many SMs (clusters of 4: 24.0 and 5.2 us); its CTAs exchange their best through
// distributed shared memory.  The division is needed only for an entry that may win: fl(w / e) >
// best implies w >= fl(best * e), one product and a comparison, and a thread's best rises only
// O(log) times over its entries.  Registers are held to 64, which four CTAs to an SM need: at 92 the
// 64 requests take 27 us.
#include <cooperative_groups.h>

#include <algorithm>
#include <utility>

#include "kda_common.cuh"
#include "kda_paged.cuh"

namespace kda {
namespace {

namespace cg = cooperative_groups;
constexpr int kVerifyCluster = 8;

struct Best {
    float race;
    int32_t at;
};
__device__ __forceinline__ void offer(Best& b, float w, float e, int v) {
    if (w > 0.f && w >= __fmul_rn(b.race, e)) {
        const float r = __fdiv_rn(w, e);
        if (r > b.race) {  // entries come in rising order: a tie stays with the earlier one
            b.race = r;
            b.at = v;
        }
    }
}
// Rising with the race, and for equal races with the lower index.  Races are >= 0.
__device__ __forceinline__ uint64_t key_of(const Best& b) {
    return (uint64_t)__float_as_uint(b.race) << 32 | (uint32_t)~b.at;
}

__device__ __forceinline__ void load4(float (&x)[4], const float* p) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void load4(float (&x)[4], const __nv_bfloat16* p) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xffff0000u);
}

// This thread's best over its share of the vocabulary.  skip: an entry whose weight is 0 (-1:
// none).  kQ: weights are max(p - q, 0).
template <typename T, bool kQ, bool kVec>
__device__ __forceinline__ Best race(const T* __restrict__ p, const T* __restrict__ q,
                                     const float* __restrict__ e, int vocab, int skip, int at,
                                     int threads) {
    Best b = {0.f, 0};
    if (kVec) {
        constexpr int kU = 2;  // (1: 20.2 us for the 64 requests above, 3: 25.4, by registers)
        const int quads = vocab >> 2;
        for (int i = at; i < quads; i += threads * kU) {
            float x[kU][4], y[kU][4], z[kU][4];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int j = i + u * threads;
                if (j < quads) {
                    load4(x[u], p + 4 * (int64_t)j);
                    if (kQ) load4(y[u], q + 4 * (int64_t)j);
                    load4(z[u], e + 4 * (int64_t)j);
                }
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int j = i + u * threads;
                if (j < quads)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int v = 4 * j + c;
                        offer(b, v == skip ? 0.f : kQ ? x[u][c] - y[u][c] : x[u][c], z[u][c], v);
                    }
            }
        }
    } else {
        constexpr int kU = 8;
        for (int i = at; i < vocab; i += threads * kU) {
            float x[kU], y[kU], z[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int v = i + u * threads;
                if (v < vocab) {
                    x[u] = io<T>::to_f(p[v]);
                    if (kQ) y[u] = io<T>::to_f(q[v]);
                    z[u] = e[v];
                }
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int v = i + u * threads;
                if (v < vocab) offer(b, v == skip ? 0.f : kQ ? x[u] - y[u] : x[u], z[u], v);
            }
        }
    }
    return b;
}

// Is some weight of the residual in this thread's share positive?
template <typename T, bool kQ>
__device__ __forceinline__ bool any_left(const T* p, const T* q, int vocab, int fallen, int at, int threads) {
#pragma unroll 1
    for (int v = at; v < vocab; v += threads) {
        const float x = io<T>::to_f(p[v]);
        if (kQ ? x - io<T>::to_f(q[v]) > 0.f : v != fallen && x > 0.f) return true;
    }
    return false;
}

template <typename T, bool kQ, bool kVec, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
verify_kernel(const VerifyArgs a, int* status) {
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ uint64_t warp_best[kThreads / 32];
    __shared__ uint64_t cta_best[3][kVerifyCluster];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = blockIdx.y, ctas = gridDim.x, rank = blockIdx.x;
    const int64_t c0 = a.cu[n], c1 = a.cu[n + 1];
    const int run = (int)(c1 - c0);
    if (c0 < 0 || run <= 0 || c1 > a.total_tokens) {  // the same for the whole cluster
        if (rank == 0 && tid == 0) {
            if (run != 0 || c0 < 0 || c1 > a.total_tokens) report_status(status, KDA_ERR_INVALID_ARG);
            a.commit[n] = 0;
            a.next[n] = -1;
        }
        return;
    }
    // the other CTAs' shared memory is written below, once all of them run
    auto started = cluster.barrier_arrive();
    const T* p = static_cast<const T*>(a.p);
    const T* q = static_cast<const T*>(a.q);
    // how many drafts hold, by every warp for itself: 32 rows at a time, the first that falls
    int took = run - 1, fallen = -1;
    for (int i0 = 0; i0 < run - 1; i0 += 32) {
        const int i = i0 + lane;
        bool falls = false;
        int x = 0;
        if (i < run - 1) {
            x = a.tokens[c0 + i + 1];
            if (x < 0 || x >= a.vocab) {
                falls = true;
                x = -1;
                report_status(status, KDA_ERR_INVALID_ARG);
            } else {
                const int64_t at = (c0 + i) * a.vocab + x;
                const float px = io<T>::to_f(p[at]), qx = kQ ? io<T>::to_f(q[at]) : 1.f;
                falls = !(__fmul_rn(a.uniform[c0 + i], qx) < px);
            }
        }
        const uint32_t m = __ballot_sync(~0u, falls);
        if (m) {
            const int j = __ffs(m) - 1;
            took = i0 + j;
            fallen = __shfl_sync(~0u, x, j);
            break;
        }
    }
    const bool fell = took < run - 1;
    const T* pr = p + (c0 + took) * a.vocab;
    const T* qr = kQ ? q + (c0 + took) * a.vocab : nullptr;
    const float* er = a.noise + (int64_t)n * a.vocab;
    const int at = rank * kThreads + tid, threads = ctas * kThreads;

    // Pass 0 is the race.  Where it leaves nothing of a fallen draft's residual, either every race was
    // zero (infinite noise, w / e below the smallest number) and they all tie, or the residual is zero
    // everywhere and the race goes over p: pass 1 looks whether some weight is positive, pass 2 races.
    uint64_t best = 0;
    for (int pass = 0; pass < 3; ++pass) {
        uint64_t k;
        if (pass == 1) {
            k = any_left<T, kQ>(pr, qr, a.vocab, fallen, at, threads) ? ~0ull : 0;
        } else {
            Best b;
            if (kQ && fell && pass == 0)
                b = race<T, true, kVec>(pr, qr, er, a.vocab, -1, at, threads);
            else
                b = race<T, false, kVec>(pr, nullptr, er, a.vocab,
                                         !kQ && fell && pass == 0 ? fallen : -1, at, threads);
            k = key_of(b);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) k = max(k, __shfl_xor_sync(~0u, k, d));
        if (lane == 0) warp_best[warp] = k;
        __syncthreads();
        if (pass == 0) cluster.barrier_wait(std::move(started));
        if (warp == 0) {
            k = lane < kThreads / 32 ? warp_best[lane] : 0;
#pragma unroll
            for (int d = 16; d; d >>= 1) k = max(k, __shfl_xor_sync(~0u, k, d));
            // every CTA gets every CTA's best
            if (lane < ctas) *cluster.map_shared_rank(&cta_best[pass][rank], lane) = k;
        }
        cluster.sync();
        best = 0;
        for (int c = 0; c < ctas; ++c) best = max(best, cta_best[pass][c]);
        if (!fell || (best >> 32) != 0) break;
    }
    // (pass 1's all ones say token 0, as ties do)
    const int token = (best >> 32) != 0 ? (int)~(uint32_t)best : 0;
    if (rank == 0) {
        if (tid == 0) {
            a.commit[n] = took + 1;
            a.next[n] = token;
        }
        for (int i = tid; i < run; i += kThreads)
            a.out[c0 + i] = i < took ? a.tokens[c0 + i + 1] : i == took ? token : -1;
    }
}

template <typename T, int kThreads>
cudaError_t launch_typed(const VerifyArgs& a, int* status, cudaStream_t stream) {
    const auto aligned = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    const bool vec = a.vocab % 4 == 0 && aligned(a.p) && aligned(a.q) && aligned(a.noise);
    void (*kernel)(const VerifyArgs, int*) =
        a.q ? (vec ? verify_kernel<T, true, true, kThreads> : verify_kernel<T, true, false, kThreads>)
            : (vec ? verify_kernel<T, false, true, kThreads> : verify_kernel<T, false, false, kThreads>);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kVerifyCluster, a.num_seqs);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kVerifyCluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, status);
}

}  // namespace

cudaError_t launch_verify_draft(const VerifyArgs& a, int* status, cudaStream_t stream) {
    // Up to one wave of clusters of 512-thread CTAs (two to an SM; 36 clusters run at once, 38 do not,
    // as a cluster does not span the SMs that other clusters leave over) a thread's chain of loads is
    // half as long: 131,072 fp32 entries, one request 6.6 us (8.7 with 256 threads), 28 requests 12.4
    // (15.1), 36 13.1 (15.6), but 38 19.5 (16.0) and 64 22.1 (18.4); 32,000 entries 5.4 (5.7) at 36.
    const bool few = (a.num_seqs + 2) * kVerifyCluster <= kPlanSMs * 2;
    if (a.dtype == KDA_BF16)
        return few ? launch_typed<__nv_bfloat16, 512>(a, status, stream)
                   : launch_typed<__nv_bfloat16, 256>(a, status, stream);
    return few ? launch_typed<float, 512>(a, status, stream) : launch_typed<float, 256>(a, status, stream);
}

}  // namespace kda
