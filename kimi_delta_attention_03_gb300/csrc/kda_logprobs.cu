// kda_logprobs.cu — log probabilities of given tokens, entropies and likeliest alternatives of rows
// of vocabulary logits.
//
//     y = s x,  m = max x,  z = sum_v e_v,  e_v = exp((x_v - m) s)
//     log p(token) = (x_token - m) s - ln z       entropy = ln z - sum_v e_v (x_v - m) s / z
//     alternatives: the k largest x, the lowest index first among equals, with their log p
//
// One pass: the sums run with a reference of the thread's own (kda_vocab.cuh), and each thread keeps
// the maximum of every batch of vectors that it has read.  The k-th largest of the threads' maxima
// bounds the k-th largest entry from below, so afterwards only the batches whose maximum reaches it
// are read again (about k of them, from L2) and their entries that reach it are the candidates: k and
// a few more, unless many entries are equal or sorted.  Then the k-th largest of the collected ones is
// a better bound, and collecting is repeated with that; each round leaves out all but k of those
// that it had collected, so it ends.  Candidates are ordered by counting the larger ones.
#include <cooperative_groups.h>

#include "kda_vocab.cuh"

namespace kda {
namespace {

namespace cg = cooperative_groups;
using namespace vocab;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kU = 4;            // vectors of a batch
constexpr int kSlots = 16;       // batch maxima that a thread keeps (neighbours share where it has more)
constexpr int kCand = 1024;      // candidates collected at a time
constexpr int kOrder = 256;      // candidates ordered by counting
constexpr int kMaxCluster = 8;

// Rising with the value, -0 as 0; -inf is kOrdNone, NaN above all.
constexpr uint32_t kOrdNone = 0x007fffffu;
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t key_of(float x, int v) {
    return (uint64_t)ordered(x) << 32 | (uint32_t)~v;
}

struct Shared {
    uint16_t slot[kSlots][kThreads];  // upper halves of the ordered batch maxima
    uint64_t cand[kCand];
    uint64_t list[kMaxTop];                     // this CTA's largest, falling
    uint64_t gather[kMaxCluster][kMaxTop];      // rank 0: every CTA's
    float sums[kMaxCluster][3];                 // rank 0: every CTA's m, z, t
    int32_t listed[kMaxCluster];
    float red_m[kWarps], red_z[kWarps], red_t[kWarps];
    int32_t count;
};

__device__ __forceinline__ uint4 load_vec(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// A CTA's part of a row: vectors [v0, v1), and (rank 0) the entries beside the whole vectors.
template <typename T>
struct Part {
    static constexpr int kVec = Row<T>::kVec;
    const T* row;
    const uint4* body;
    int head, vocab, edges;
    int v0, v1, batches, shift;
    __device__ __forceinline__ Part(const T* row_, int vocab_, int rank, int ctas)
        : row(row_), vocab(vocab_) {
        const Cut c = cut_row(row, vocab);
        head = c.head;
        body = reinterpret_cast<const uint4*>(row + head);
        v0 = (int)(c.body * rank / ctas);
        v1 = (int)(c.body * (rank + 1) / ctas);
        edges = rank == 0 ? c.head + c.tail : 0;
        batches = max((v1 - v0 + kThreads * kU - 1) / (kThreads * kU), 1);
        shift = 0;
        while ((batches - 1) >> shift >= kSlots) ++shift;
    }
    __device__ __forceinline__ int edge(int i) const { return i < head ? i : vocab - edges + i; }
    __device__ __forceinline__ int first(int b) const { return v0 + b * kThreads * kU + (int)threadIdx.x; }
    __device__ __forceinline__ void load(uint4 (&r)[kU], int b) const {
        const int j = first(b);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const uint32_t none = Row<T>::kNone;
            r[u] = make_uint4(none, none, none, none);
            if (j + u * kThreads < v1) r[u] = load_vec(body + j + u * kThreads);
        }
    }
};

__device__ __forceinline__ void offer(Shared& sm, uint64_t bound, float x, int v) {
    const uint64_t k = key_of(x, v);
    if (k >= bound) {
        const int at = atomicAdd(&sm.count, 1);
        if (at < kCand) sm.cand[at] = k;
    }
}
// The k-th largest of sm.cand[0 .. n), n >= k.
__device__ __forceinline__ uint64_t kth_candidate(const Shared& sm, int n, int k) {
    uint64_t mine[kCand / kThreads], kth = 0;
#pragma unroll
    for (int i = 0; i < kCand / kThreads; ++i) {
        const int at = threadIdx.x + i * kThreads;
        mine[i] = at < n ? sm.cand[at] : 0;
    }
#pragma unroll 1
    for (int b = 63; b >= 0; --b) {
        const uint64_t t = kth | 1ull << b;
        int count = 0;
#pragma unroll
        for (int i = 0; i < kCand / kThreads; ++i) count += __syncthreads_count(mine[i] >= t);
        if (count >= k) kth = t;
    }
    return kth;
}

// The part's k largest above -inf into sm.list, falling; returns how many.
template <typename T>
__device__ __forceinline__ int largest(Shared& sm, const Part<T>& part, int k, float top) {
    const int tid = threadIdx.x, slots = ((part.batches - 1) >> part.shift) + 1;
    const uint32_t mine = ordered(top) >> 16;
    uint32_t low = 0;  // largest value that k threads' maxima reach, by their upper halves
#pragma unroll 1
    for (int b = 15; b >= 0; --b) {
        const uint32_t t = low | 1u << b;
        if (__syncthreads_count(mine >= t) >= k) low = t;
    }
    uint64_t bound = max((uint64_t)low << 48, (uint64_t)(kOrdNone + 1) << 32);
    int n;
    while (true) {
        if (tid == 0) sm.count = 0;
        __syncthreads();
        for (int s = 0; s < slots; ++s) {
            if (sm.slot[s][tid] < (uint32_t)(bound >> 48)) continue;
            if (s == 0 && tid < part.edges) {
                const int v = part.edge(tid);
                offer(sm, bound, io<T>::to_f(part.row[v]), v);
            }
            const int last = min((s + 1) << part.shift, part.batches);
            for (int b = s << part.shift; b < last; ++b) {
                uint4 r[kU];
                part.load(r, b);
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int v = part.head + (part.first(b) + u * kThreads) * Part<T>::kVec;
                    const uint32_t w[4] = {r[u].x, r[u].y, r[u].z, r[u].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (sizeof(T) == 2) {
                            const float2 x = unpack(w[i]);
                            offer(sm, bound, x.x, v + 2 * i);
                            offer(sm, bound, x.y, v + 2 * i + 1);
                        } else {
                            offer(sm, bound, __uint_as_float(w[i]), v + i);
                        }
                    }
                }
            }
        }
        __syncthreads();
        n = sm.count;
        if (n <= kOrder) break;
        bound = kth_candidate(sm, min(n, kCand), k);
        __syncthreads();  // sm.count and sm.cand are read
    }
    if (tid < n) {
        const uint64_t me = sm.cand[tid];
        int rank = 0;
        for (int i = 0; i < n; ++i) rank += sm.cand[i] > me;
        if (rank < k) sm.list[rank] = me;
    }
    return min(n, k);
}

template <typename T, bool kTop>
__global__ void __launch_bounds__(kThreads, 3) logprobs_kernel(const LogprobArgs a, int* status) {
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ Shared sm;
    const int tid = threadIdx.x, ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int64_t row = blockIdx.x / ctas;
    const int token = a.tokens ? a.tokens[row] : 0;
    const float s = a.inv_temperature ? a.inv_temperature[row] : 1.f, c = s * kLog2e;
    const bool asked = token >= 0 && token < a.vocab, sane = s > 0.f && c < INFINITY;
    if (!asked || !sane) {  // the same for the whole cluster
        if (rank == 0) {
            const float none = __int_as_float(0x7fffffff);
            if (tid == 0) {
                if (token >= a.vocab) report_status(status, KDA_ERR_INVALID_ARG);
                if (a.logprobs) a.logprobs[row] = asked ? none : 0.f;
                a.entropy[row] = asked ? none : 0.f;
            }
            for (int i = tid; i < a.top_k; i += kThreads) {
                a.top_ids[row * a.top_k + i] = -1;
                a.top_logprobs[row * a.top_k + i] = asked ? none : -INFINITY;
            }
        }
        return;
    }
    // rank 0's shared memory is written below, once all CTAs run
    cluster_arrive();
    const T* x = static_cast<const T*>(a.logits) + row * a.stride;
    const Part<T> part(x, a.vocab, rank, ctas);
    const float chosen = rank == 0 && tid == 0 && a.tokens ? io<T>::to_f(x[token]) : 0.f;
    Online o;
    float batch_top = -INFINITY;
    if (tid < part.edges) {
        batch_top = io<T>::to_f(x[part.edge(tid)]);
        add_one<true>(o, batch_top, c);
    }
#pragma unroll 1
    for (int b = 0; b < part.batches; ++b) {
        uint4 r[kU];
        part.load(r, b);
        batch_top = max_nan(batch_top, add_vectors<T, true>(o, r, c));
        if (kTop && ((b + 1) & ((1 << part.shift) - 1)) == 0) {
            sm.slot[b >> part.shift][tid] = (uint16_t)(ordered(batch_top) >> 16);
            batch_top = -INFINITY;
        }
    }
    if (kTop && (part.batches & ((1 << part.shift) - 1)) != 0)
        sm.slot[(part.batches - 1) >> part.shift][tid] = (uint16_t)(ordered(batch_top) >> 16);
    // the CTA's sums about its maximum
    float m = block_max<kWarps>(o.top, sm.red_m);
    const float d = octaves(o.m, m, c), f = sm100::ex2_approx(d), zt = o.z.x + o.z.y;
    float z = block_sum<kWarps>(zt * f, sm.red_z);
    float t = block_sum<kWarps>((o.t.x + o.t.y + zt * d) * f, sm.red_t);
    int n = 0;
    if constexpr (kTop) n = largest(sm, part, a.top_k, o.top);
    cluster_wait();
    if (ctas > 1) {
        if (tid == 0) {
            float* to = cluster.map_shared_rank(&sm.sums[rank][0], 0);
            to[0] = m;
            to[1] = z;
            to[2] = t;
            *cluster.map_shared_rank(&sm.listed[rank], 0) = n;
        }
        __syncthreads();  // sm.list
        if (tid < n) *cluster.map_shared_rank(&sm.gather[rank][tid], 0) = sm.list[tid];
        cluster_arrive();
        cluster_wait();
        if (rank != 0) return;
        m = -INFINITY;
        for (int r = 0; r < ctas; ++r) m = max_nan(m, sm.sums[r][0]);
        z = t = 0.f;
        for (int r = 0; r < ctas; ++r) {
            const float dr = octaves(sm.sums[r][0], m, c), fr = sm100::ex2_approx(dr);
            z += sm.sums[r][1] * fr;
            t += (sm.sums[r][2] + sm.sums[r][1] * dr) * fr;
        }
    } else {
        __syncthreads();  // sm.list
    }
    const bool fine = z > 0.f && z < INFINITY;  // else NaN or inf, or nothing above -inf
    const float none = __int_as_float(0x7fffffff), ln_z = logf(z);
    if (tid == 0) {
        // (the clamps take off what approximate exponentials leave beyond the range)
        if (a.logprobs) a.logprobs[row] = fine ? fminf((chosen - m) * s - ln_z, 0.f) : none;
        a.entropy[row] = fine ? fmaxf(ln_z - t / z * kLn2, 0.f) : none;
    }
    if constexpr (kTop) {
        const auto put = [&](int at, uint64_t key) {
            a.top_ids[row * a.top_k + at] = fine ? (int)~(uint32_t)key : -1;
            a.top_logprobs[row * a.top_k + at] =
                fine ? fminf((from_ordered((uint32_t)(key >> 32)) - m) * s - ln_z, 0.f) : none;
        };
        int total = n;
        if (ctas == 1) {
            if (tid < n) put(tid, sm.list[tid]);
        } else {
            total = 0;
            for (int r = 0; r < ctas; ++r) total += sm.listed[r];
            // an entry's place: its place in its own list and the larger ones in the others
            for (int i = tid; i < ctas * kMaxTop; i += kThreads) {
                const int r = i / kMaxTop, at = i % kMaxTop;
                if (at >= sm.listed[r]) continue;
                const uint64_t me = sm.gather[r][at];
                int place = at;
                for (int q = 0; q < ctas; ++q) {
                    if (q == r) continue;
                    int lo = 0, hi = sm.listed[q];
                    while (lo < hi) {
                        const int mid = (lo + hi) >> 1;
                        if (sm.gather[q][mid] > me) lo = mid + 1; else hi = mid;
                    }
                    place += lo;
                }
                if (place < a.top_k) put(place, me);
            }
        }
        for (int i = total + tid; i < a.top_k; i += kThreads) {
            a.top_ids[row * a.top_k + i] = -1;
            a.top_logprobs[row * a.top_k + i] = fine ? -INFINITY : none;
        }
    }
}

template <typename T, bool kTop>
cudaError_t launch_typed(const LogprobArgs& a, int ctas, int* status, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.rows * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, kTop>, a, status);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, int* status, cudaStream_t stream) {
    // few rows are split over a cluster, as long as that fills SMs and a thread has a batch
    const int64_t bytes = (int64_t)a.vocab * (a.dtype == KDA_BF16 ? 2 : 4);
    int ctas = 1;
    while (ctas < kMaxCluster && a.rows * ctas * 2 <= 3 * kPlanSMs && bytes / (ctas * 2) >= kThreads * 16)
        ctas *= 2;
    if (a.dtype == KDA_BF16)
        return a.top_k ? launch_typed<__nv_bfloat16, true>(a, ctas, status, stream)
                       : launch_typed<__nv_bfloat16, false>(a, ctas, status, stream);
    return a.top_k ? launch_typed<float, true>(a, ctas, status, stream)
                   : launch_typed<float, false>(a, ctas, status, stream);
}

}  // namespace kda
