// kda_logprobs.cu — log probabilities of given tokens, entropies and likeliest alternatives of rows
// of vocabulary logits.
//
//     y = s x,  m = max x,  z = sum_v e_v,  e_v = exp((x_v - m) s)
//     log p(token) = (x_token - m) s - ln z       entropy = ln z - sum_v e_v (x_v - m) s / z
//     alternatives: the k largest x, the lowest index first among equals, with their log p
//
// One pass: the sums run with a reference of the thread's own (kda_vocab.cuh), and each thread keeps
// the maxima of the batches of vectors that it has read.  The k-th largest of the threads' maxima
// bounds the k-th largest entry from below, so afterwards only a thread's batch whose maximum reaches
// that bound is read again (about k of them, from L2), and the entries that reach it are the
// candidates: k and a few more, unless many entries are equal or sorted.  Then the k-th largest of the
// collected ones is a better bound, and collecting is repeated with that; each round leaves out all but
// k of those that it had collected, so it ends.  Candidates are ordered by counting the larger ones.
//
// What bounds it: long rows the memory (4,096 rows of 131,072 bf16 entries, one alternative: 163 us, 97% of
// the measured copy bandwidth).  With many alternatives of shorter rows it is the chain after the stream: 2,048
// rows of 50,001 with 64 take 53 us (57%), 38 without the alternatives, of which the bound, collecting and
// ordering take about a third each (54 when one candidate was compared with one other at a time).  A search for
// the bound bit by bit over barriers, and whole threads that read their entries again, took 102 us.  64 rows of
// 131,072 with 20 take 9.5 us and one row of 32,000 5.6, which is launch and latency.  Rows of equal entries cost
// more: 2,048 of 131,072 at a mask's value, four tokens beside it, 20 alternatives, take 224 us in bf16 (94 without a
// mask).  In fp32 the bound is the upper half of a value, so that leaving out later equal entries works only for
// values whose ordered lower half is zeros: 814 us at the type's lowest value, 1,140 at -1e9, -1e4 or -65504 (177
// without a mask, 169 at -inf).
#include <cooperative_groups.h>

#include "kda_vocab.cuh"

namespace kda {
namespace {

namespace cg = cooperative_groups;
using namespace vocab;

constexpr int kSlots = 16;       // maxima that a thread keeps (neighbouring batches share one where there are more)
constexpr int kCand = 1024;      // candidates collected at a time
constexpr int kOrder = 256;      // candidates ordered by counting
constexpr int kBins = 256;       // upper halves below the maximum among which the bound is looked for at first
constexpr int kMany = 512;       // maxima queued above which many entries are equal
constexpr int kMaxCluster = 8;
static_assert(kMaxCluster * kMaxTop <= kCand, "the lists of a cluster's CTAs are candidates once more");

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

template <int kThreads>
struct Shared {
    uint16_t slot[kSlots][kThreads];            // upper halves of the ordered maxima
    uint16_t queue[kSlots * kThreads];          // of them, those to read again: slot * kThreads + thread
    __align__(16) uint64_t cand[kCand];
    uint64_t gather[kMaxCluster][kMaxTop];      // rank 0: every CTA's largest, falling
    float4 joined[kMaxCluster];                 // rank 0: every CTA's m, z, t, how many largest
    float3 sums[kThreads / 32];
    __align__(16) int32_t bins[kBins];
    int32_t queued, count;
};

// The k-th largest of sm.cand[0 .. n), n >= k, bit by bit from the first in which they differ.  (The bins are not
// needed any more and count here.)
template <int kThreads>
__device__ __noinline__ uint64_t kth_candidate(Shared<kThreads>& sm, int n, int k) {
    constexpr int kMine = kCand / kThreads;
    const int tid = threadIdx.x;
    const uint64_t any = sm.cand[0];
    uint64_t mine[kMine], differ = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int at = tid + i * kThreads;
        mine[i] = at < n ? sm.cand[at] : 0;
        if (at < n) differ |= mine[i] ^ any;
    }
    if (tid < 66) sm.bins[tid] = 0;
    __syncthreads();
    const uint32_t high = __reduce_or_sync(~0u, (uint32_t)(differ >> 32)), below = __reduce_or_sync(~0u, (uint32_t)differ);
    if (tid % 32 == 0) {
        atomicOr(&sm.bins[64], (int)high);
        atomicOr(&sm.bins[65], (int)below);
    }
    __syncthreads();
    differ = (uint64_t)(uint32_t)sm.bins[64] << 32 | (uint32_t)sm.bins[65];
    const int bits = 64 - __clzll((long long)differ);
    uint64_t kth = bits == 64 ? 0 : any >> bits << bits;
#pragma unroll 1
    for (int b = bits - 1; b >= 0; --b) {
        const uint64_t t = kth | 1ull << b;
        int count = 0;
#pragma unroll
        for (int i = 0; i < kMine; ++i) count += mine[i] >= t;
        count = __reduce_add_sync(~0u, count);
        if (tid % 32 == 0 && count) atomicAdd(&sm.bins[b], count);
        __syncthreads();
        if (sm.bins[b] >= k) kth = t;
    }
    return kth;
}
// The largest value that k threads' maxima reach, by upper halves: from the counts below the CTA's maximum,
// every warp for itself; where those are too few (maxima far apart), bit by bit.
template <int kThreads>
__device__ __forceinline__ uint32_t reached_by(Shared<kThreads>& sm, int k, uint32_t mine, uint32_t most) {
    if (most - mine < kBins) atomicAdd(&sm.bins[most - mine], 1);
    __syncthreads();
    const int lane = threadIdx.x & 31;
    static_assert(kBins == 256, "a lane has eight");
    const int4 a = reinterpret_cast<const int4*>(sm.bins)[2 * lane], b = reinterpret_cast<const int4*>(sm.bins)[2 * lane + 1];
    const int n[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    int upto = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) upto += n[i];
    int left = -upto;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(~0u, upto, d);
        if (lane >= d) upto += y;
    }
    const uint32_t who = __ballot_sync(~0u, upto >= k);
    if (who) {
        left += upto;
        int bin = lane * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            left += n[i];
            if (left < k) ++bin;
        }
        return most - __shfl_sync(~0u, bin, __ffs(who) - 1);
    }
    uint32_t low = 0;
#pragma unroll 1
    for (int i = 15; i >= 0; --i) {
        const uint32_t t = low | 1u << i;
        if (__syncthreads_count(mine >= t) >= k) low = t;
    }
    return low;
}
template <int kThreads>
__device__ __forceinline__ void offer(Shared<kThreads>& sm, uint64_t bound, float x, int v) {
    const uint64_t k = key_of(x, v);
    if (k >= bound) {
        const int at = atomicAdd(&sm.count, 1);
        if (at < kCand) sm.cand[at] = k;
    }
}
// The part's candidates into sm.cand: among them its k largest above -inf.  Returns how many, at most kOrder.
template <typename T, int kThreads>
__device__ __forceinline__ int candidates(Shared<kThreads>& sm, const T* row, const Part<T>& part, int batches, int shift,
                                          int k, uint32_t mine, uint32_t low) {
    constexpr int kBatch = kThreads * kU;
    const int tid = threadIdx.x, whole = part.whole();
    const uint4* const body = reinterpret_cast<const uint4*>(row + part.body0);
    const int slots = ((batches - 1) >> shift) + 1;
    // (of bf16 the value itself: the lower half is zeros, or ones below zero)
    const uint32_t value = low << 16 | (sizeof(T) == 2 && !(low & 0x8000u) ? 0xffffu : 0u);
    uint64_t bound = (uint64_t)max(value, kOrdNone + 1) << 32;
    bool narrowed = false;
    while (true) {  // (sm.queued and sm.count are 0)
        const uint32_t reach = (uint32_t)(bound >> 48), upto = ~(uint32_t)bound;  // upto: indices of equal entries
        if (mine >= reach) {
            if (part.edge(tid) >= 0) offer(sm, bound, io<T>::to_f(row[part.edge(tid)]), part.edge(tid));
            for (int s = 0; s < slots; ++s) {
                const uint32_t top = sm.slot[s][tid];
                if (top < reach) continue;
                // a bf16 maximum that equals the bound, behind the indices that count
                if (sizeof(T) == 2 && top == reach && part.body0 + ((s << shift) * kBatch + tid) * Row<T>::kVec > upto)
                    continue;
                sm.queue[atomicAdd(&sm.queued, 1)] = (uint16_t)(s * kThreads + tid);
            }
        }
        __syncthreads();
        if (sm.queued > kMany && !narrowed) {
            // Equal entries by the thousand (a mask's value, with fewer tokens than alternatives beside it): the
            // first slots in which k maxima reach the bound hold k entries, so later ones that equal it do not count.
            narrowed = true;
            int n = 0, s = 0;
            for (; s < slots; ++s) {
                n += __syncthreads_count(sm.slot[s][tid] >= reach);
                if (n >= k) break;
            }
            if (s + 1 < slots) {
                bound |= ~(uint32_t)(part.body0 + ((s + 1) << shift) * kBatch * Row<T>::kVec - 1);
                for (int i = tid; i < kOrder; i += kThreads) sm.cand[i] = 0;
                if (tid == 0) sm.queued = sm.count = 0;
                __syncthreads();
                continue;
            }
        }
        // a lane to a vector; those of a slot's further batches one after another
        const uint32_t at_least = (uint32_t)(bound >> 32);
        const int items = sm.queued * kU;
        for (int i0 = tid; i0 < items; i0 += 2 * kThreads) {
            for (int b = 0; b < 1 << shift; ++b) {
                uint4 r[2];
                int j[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {  // two under way
                    const int i = i0 + h * kThreads, q = i < items ? sm.queue[i / kU] : 0;
                    j[h] = ((q / kThreads << shift) + b) * kBatch + q % kThreads + i % kU * kThreads;
                    if (i >= items) j[h] = whole;
                    r[h] = make_uint4(Row<T>::kNone, Row<T>::kNone, Row<T>::kNone, Row<T>::kNone);
                    if (j[h] < whole) r[h] = load_vec(body + j[h], drop_policy());
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t in = 0;
                    // (behind the indices that count an entry has to be larger)
                    const float least = from_ordered(at_least + (part.body0 + j[h] * Row<T>::kVec > upto));
                    const uint32_t w[4] = {r[h].x, r[h].y, r[h].z, r[h].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if constexpr (sizeof(T) == 2) {
                            const float2 x = unpack(w[k]);
                            in |= (uint32_t)!(x.x < least) << (2 * k) | (uint32_t)!(x.y < least) << (2 * k + 1);
                        } else {
                            in |= (uint32_t)!(__uint_as_float(w[k]) < least) << k;
                        }
                    }
                    for (; in; in &= in - 1) {
                        const int e = __ffs(in) - 1, k = sizeof(T) == 2 ? e >> 1 : e;
                        const uint32_t word = k & 2 ? (k & 1 ? w[3] : w[2]) : (k & 1 ? w[1] : w[0]);
                        const float x = __uint_as_float(sizeof(T) == 4 ? word : e & 1 ? word & 0xffff0000u : word << 16);
                        offer(sm, bound, x, part.body0 + j[h] * Row<T>::kVec + e);
                    }
                }
            }
        }
        __syncthreads();
        const int n = sm.count;
        if (n <= kOrder) return n;
        bound = kth_candidate(sm, min(n, kCand), k);
        __syncthreads();  // what follows is read
        for (int i = tid; i < kOrder; i += kThreads) sm.cand[i] = 0;
        if (tid == 0) sm.queued = sm.count = 0;
        __syncthreads();
    }
}
// sm.cand[0 .. n), n at most kOrder, by their places in falling order: four lanes to two candidates, which they
// compare with two others at a time.  (Behind the last there are zeros, below every key.)
template <int kThreads, typename Put>
__device__ __forceinline__ void in_order(const Shared<kThreads>& sm, int n, Put put) {
    const int tid = threadIdx.x;
    constexpr int kHalf = kThreads / 4;
    const ulonglong2* const pairs = reinterpret_cast<const ulonglong2*>(sm.cand);
    for (int i0 = 0; i0 < n; i0 += 2 * kHalf) {
        const int i = i0 + tid / 4;
        const uint64_t me = sm.cand[i], other = sm.cand[i + kHalf];
        int place = 0, place1 = 0;
#pragma unroll 2
        for (int j = tid % 4; 2 * j < n; j += 4) {
            const ulonglong2 c = pairs[j];
            place += (c.x > me) + (c.y > me);
            place1 += (c.x > other) + (c.y > other);
        }
        place |= place1 << 16;
        place += __shfl_xor_sync(~0u, place, 1);
        place += __shfl_xor_sync(~0u, place, 2);
        if (tid % 4 == 0 && me) put(place & 0xffff, me);
        if (tid % 4 == 1 && other) put(place >> 16, other);
    }
}

template <typename T, bool kTop, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) logprobs_kernel(const LogprobArgs a, int* status) {
    cg::cluster_group cluster = cg::this_cluster();
    constexpr int kWarps = kThreads / 32, kBatch = kThreads * kU;
    __shared__ __align__(16) Shared<kThreads> sm;
    const int tid = threadIdx.x, ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int64_t row = blockIdx.x / ctas;
    const int token = a.tokens ? a.tokens[row] : 0;
    const float s = a.inv_temperature ? a.inv_temperature[row] : 1.f, c = s * kLog2e;
    // (before it is known whether the row is asked for: as long as that takes, so does its first batch)
    const T* x = static_cast<const T*>(a.logits) + row * a.stride;
    const Part<T> part(x, a.vocab, rank, ctas);
    const int whole = part.whole(), batches = max((whole + kBatch - 1) / kBatch, 1);
    const uint4* const body = reinterpret_cast<const uint4*>(x + part.body0);
    uint4 next[kU];
    const uint64_t policy = drop_policy();
    load_batch<T, kThreads, false>(next, body, 0, whole, policy);
    if (tid == 0) fetch<kThreads>(body, 1, kAhead - 1, whole);
    const float none = __int_as_float(0x7fffffff);
    const bool asked = token >= 0 && token < a.vocab;
    if (!asked || !(s > 0.f && s <= 0x1p127f)) {  // the same for the whole cluster; above, c is beyond fp32
        if (rank == 0) {
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
    if (ctas > 1) cluster_arrive();  // rank 0's shared memory is written below, once all run
    const float chosen = rank == 0 && tid == 0 && a.tokens ? io<T>::to_f(x[token]) : 0.f;
    int shift = 0;
    while ((batches - 1) >> shift >= kSlots) ++shift;
    if constexpr (kTop) {
        for (int i = tid; i < kBins; i += kThreads) sm.bins[i] = 0;
        if (tid == 0) sm.queued = sm.count = 0;
        for (int i = tid; i < kOrder; i += kThreads) sm.cand[i] = 0;
    }
    const float lim = limit(c);
    Online o;
    if (part.edge(tid) >= 0) add_one(o, io<T>::to_f(x[part.edge(tid)]), c, lim);
    float top = -INFINITY;  // since the last slot
    if (kTop && whole == 0) sm.slot[0][tid] = kOrdNone >> 16;
    stream<T, kThreads, false, false, true>(body, whole, policy, next, [&](const uint4 (&r)[kU], int j) {
        top = max_nan(top, add_vectors<T, true>(o, r, c, lim));
        const int b = j / kBatch;
        if (kTop && (((b + 1) & ((1 << shift) - 1)) == 0 || b + 1 == batches)) {
            sm.slot[b >> shift][tid] = (uint16_t)(ordered(top) >> 16);
            top = -INFINITY;
        }
    });
    float3 q = warp_sums<true>(o, c, lim);  // (m, z, t)
    if (tid % 32 == 0) sm.sums[tid / 32] = q;
    __syncthreads();
    q = lane_sums<true>(sm.sums[tid % kWarps], kWarps, c);
    if (fabsf(q.x) >= lim && fabsf(q.x) < INFINITY) {
        __syncthreads();
        q = far_sums<T, kThreads, true>(x, part, nullptr, 0, q.x, c);
        if (tid % 32 == 0) sm.sums[tid / 32] = q;
        __syncthreads();
        q = lane_sums<true>(sm.sums[tid % kWarps], kWarps, c);
    }
    int n = 0;
    if constexpr (kTop) {
        const uint32_t mine = ordered(o.top) >> 16;
        n = candidates(sm, x, part, batches, shift, a.top_k, mine, reached_by(sm, a.top_k, mine, ordered(q.x) >> 16));
    }
    if (ctas > 1) {
        cluster_wait();
        if constexpr (kTop)
            in_order(sm, n, [&](int place, uint64_t key) {
                if (place < a.top_k) *cluster.map_shared_rank(&sm.gather[rank][place], 0) = key;
            });
        n = min(n, a.top_k);
        if (tid == 0) *cluster.map_shared_rank(&sm.joined[rank], 0) = make_float4(q.x, q.y, q.z, __int_as_float(n));
        cluster_arrive();
        cluster_wait();
        if (rank != 0) return;
        const float4 each = sm.joined[tid % ctas];
        q = lane_sums<true>(make_float3(each.x, each.y, each.z), ctas, c);
        if constexpr (kTop) {
            // The largest of the lists' k-th bounds the k-th of all; what reaches it is ordered once more.
            for (int i = tid; i < kOrder; i += kThreads) sm.cand[i] = 0;
            if (tid == 0) sm.count = 0;
            uint64_t bound = 0;
            for (int r = 0; r < ctas; ++r)
                if (__float_as_int(sm.joined[r].w) == a.top_k) bound = max(bound, sm.gather[r][a.top_k - 1]);
            while (true) {
                __syncthreads();
                for (int i = tid; i < ctas * a.top_k; i += kThreads) {
                    const int r = i / a.top_k, at = i - r * a.top_k;
                    if (at < __float_as_int(sm.joined[r].w) && sm.gather[r][at] >= bound)
                        sm.cand[atomicAdd(&sm.count, 1)] = sm.gather[r][at];
                }
                __syncthreads();
                n = sm.count;
                if (n <= kOrder) break;
                bound = kth_candidate(sm, n, a.top_k);
                __syncthreads();
                for (int i = tid; i < kOrder; i += kThreads) sm.cand[i] = 0;
                if (tid == 0) sm.count = 0;
            }
        }
    }
    const bool fine = fabsf(q.x) < INFINITY;  // else NaN or inf, or nothing above -inf
    const float ln_z = logf(q.y);
    if (tid == 0) {
        // (the clamps here and below take off what approximate exponentials leave beyond the range)
        if (a.logprobs) a.logprobs[row] = fine ? fminf(scaled(chosen, q.x, s, ln_z), 0.f) : none;
        a.entropy[row] = fine ? fmaxf(ln_z - q.z / q.y * kLn2, 0.f) : none;
    }
    if constexpr (kTop) {
        int32_t* const ids = a.top_ids + row * a.top_k;
        float* const best = a.top_logprobs + row * a.top_k;
        in_order(sm, n, [&](int place, uint64_t key) {
            if (place >= a.top_k) return;
            ids[place] = fine ? (int)~(uint32_t)key : -1;
            best[place] = fine ? fminf(scaled(from_ordered((uint32_t)(key >> 32)), q.x, s, ln_z), 0.f) : none;
        });
        for (int i = n + tid; i < a.top_k; i += kThreads) {
            ids[i] = -1;
            best[i] = fine ? -INFINITY : none;
        }
    }
}

template <typename T, bool kTop, int kThreads>
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
    cfg.numAttrs = ctas > 1;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, kTop, kThreads>, a, status);
}
template <typename T, int kThreads>
cudaError_t launch_top(const LogprobArgs& a, int ctas, int* status, cudaStream_t stream) {
    return a.top_k ? launch_typed<T, true, kThreads>(a, ctas, status, stream)
                   : launch_typed<T, false, kThreads>(a, ctas, status, stream);
}
template <typename T>
cudaError_t launch_rows(const LogprobArgs& a, int* status, cudaStream_t stream) {
    const int64_t bytes = (int64_t)a.vocab * sizeof(T);
    // Many short rows take CTAs of 128 threads, whose warps have half the joining and ordering to do: 4,096
    // rows with 20 alternatives, of 8 KB 22 us in bf16 and 20 in fp32 (256 threads: 39 and 36), 32 KB 36 and 33 (48
    // and 44), 64 KB 55 and 53 (64 and 61); without alternatives 44 and 42 at 64 KB (46 and 44).  The more
    // alternatives and the longer the row, the less: with 64 of them 51 and 47 at 32 KB (56 and 51), 75 and 72 at 64
    // KB (74 and 68), and 2,048 rows of 98 KB 55 and 53 (53 and 50; with 20 44 and 42, against 48 and 47).  Above 64
    // alternatives the threads' maxima are too few.
    if (a.rows > 4 * kPlanSMs && bytes <= 64 * 1024 && a.top_k <= 64) return launch_top<T, 128>(a, 1, status, stream);
    // Few rows are split over a cluster, as long as its CTAs are two to an SM and a thread has a vector: one row
    // of 32,000 fp32 entries takes 5.6 us on eight CTAs, 6.3 on four, 6.9 on two; but 64 rows of 131,072 bf16
    // entries 12.7 on eight and 9.5 on four.
    int ctas = 1;
    while (ctas < kMaxCluster && a.rows * ctas * 2 <= 2 * kPlanSMs && bytes / (ctas * 2) >= 4096) ctas *= 2;
    return launch_top<T, 256>(a, ctas, status, stream);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, int* status, cudaStream_t stream) {
    return a.dtype == KDA_BF16 ? launch_rows<__nv_bfloat16>(a, status, stream) : launch_rows<float>(a, status, stream);
}

}  // namespace kda
