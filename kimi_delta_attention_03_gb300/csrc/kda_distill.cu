// kda_distill.cu — distillation of rows of vocabulary logits from a teacher's top entries: losses,
// gradients for given gradients of the losses, and both in one call.
//
//     q = softmax(s x);  entries (id_i, v_i), i < K;  p_i = softmax(v)_i
//     L = sum_i p_i (log p_i - log q[id_i])                 dL/dx_v = s (M q_v - P_v)
// with P_v the sum of the p_i of token v and M = 1.  With `tail` v are log probabilities, p_i =
// exp(v_i), and r = max(0, 1 - sum p) is the mass of one more outcome, all tokens outside the entries:
//     L += r (log r - log q_r)         M = sum p + r,   dL/dx_v -= s r q_v / q_r  for v outside
//
// The tokens outside are summed by themselves, not as what the entries leave of the whole row, which
// cancels where the entries hold nearly all of it: with m_r their largest logit and z_r = sum exp((x -
// m_r) s) over them, every weight of theirs in the gradient is one factor times exp((x_v - m_r) s).
//
// Where sums and gradient are wanted at once the row is read twice, the second time right after the first and
// backwards, mostly from L2: so many rows are under way at a time as fit there.  It is asked to keep what the first
// pass reads and to drop what the second reads and writes (4,096 rows of 131,072 bf16 entries: 384 us, without that
// 413; DRAM reads 1.15 times the logits).  Where all rows fit L2 by themselves that gains less: 13.1 us and 13.2 for
// 64 such rows, 19.3 and 19.8 for 128, 30.3 and 33.7 for 256.  What was kept costs what runs next little: an addition
// over 16 or 32 MB right after is no slower, one over 48 MB takes 18.4 us instead of 16.4.  Rows of weight 0 that have
// entries are kept and not read again: with three rows in ten of them the 4,096 take 370 us, and what runs next is no
// slower.  Giving the lines back one by one (applypriority) took 3 to 8% longer for 32,000 and 50,001 entries and for
// 500 rows of 131,072, and was equal for 4,096 of those.
//
// What bounds it: memory.  2,048 such rows' losses take 77 us (92% of the measured copy bandwidth), their gradient
// 157 (96%), both of 4,096 rows 384 (82%): some 35 us less if the second pass read nothing, the rest is L2 and reads
// that miss it.  2,048 rows of 65,536 fp32 entries: 81 us (98%), 163 (97%) and 191 (83%).  Keeping parts in shared
// memory between the passes was slower: all of a part in clusters of four by a third, its last 16 or 32 KB by 2 to 3%.
// 1,000 ragged rows of 50,001, the gradient in rows of another alignment, take 48 us (52%): one wave of CTAs and a
// nearly empty second one.  64 rows of 32,000: 5.5 us, launch and latency.
#include <cooperative_groups.h>

#include "kda_vocab.cuh"

namespace kda {
namespace {

namespace cg = cooperative_groups;
using namespace vocab;

constexpr int kThreads = 256, kWarps = kThreads / 32, kBatch = kThreads * kU;
static_assert(kMaxTeacher <= kThreads, "a thread has an entry");
struct Shared {
    float4 sums[kDistillCluster];   // every CTA's sums: m_r, z_r, and those of its entries
    float2 teacher;                 // from rank 0: r and M
    int32_t ids[kMaxTeacher];
    float p[kMaxTeacher];
    float3 outside[kWarps];
    float2 entries[kWarps], given[kWarps];  // the entries' logits' sums; the teacher's values'
    int64_t mass[kWarps];
    float loss[kWarps];
    uint32_t edge_held;             // entries beside whole vectors that the teacher names
    int32_t twice;                  // some token is named more than once
};

// e^v in units of 2^-40, v at most 8: reduced by multiples of ln 2 held in three parts (Cody and Waite), then
// the Taylor series, whose first terms are kept in two parts.  Relative error about 2^-30, so that what the
// entries leave of 1 is exact to some 1e-9; doubles would do, but take these SMs 3,000 cycles here.
__device__ __forceinline__ int64_t exp_fixed(float v) {
    if (v < -30.f) return 0;
    constexpr float kHigh = 0.693359375f;                          // 9 bits: multiples are exact
    constexpr double kLow = -2.1219444005469058277e-4;             // ln 2 - kHigh
    constexpr float kMid = (float)kLow, kRest = (float)(kLow - (double)kMid);
    const float n = rintf(v * kLog2e), x = fmaf(-n, kHigh, v);     // exact
    const float y = -n * kMid, a = x + y, t = a - x;
    const float b = (x - (a - t)) + (y - t) + fmaf(-n, kMid, -y) - n * kRest;  // a + b: the reduced argument
    const float h = a * a, l = fmaf(a, a, -h);
    const float q = fmaf(a, fmaf(a, fmaf(a, fmaf(a, fmaf(a, 1.f / 362880, 1.f / 40320), 1.f / 5040), 1.f / 720), 1.f / 120), 1.f / 24);
    const float small = fmaf(h * h, q, a * h * (1.f / 6)) + (0.5f * l + b * (1.f + a + 0.5f * h));
    const int64_t one = 1ll << 40;
    const int64_t e = one + __float2ll_rn(a * (float)one) + __float2ll_rn(h * (float)(one / 2)) + __float2ll_rn(small * (float)one);
    const int by = (int)n;
    return by >= 0 ? e << by : e >> -by;
}

// f exp2((x - from) c), of a vector and of one logit.
struct Weigh {
    float from, c, f, off;
    // Octaves as fma(x, c, off); else differences first.  One that is beyond fp32 is then 2^20 octaves at least, nothing:
    // from c is 2^20 or more and from below 2^128, so that c is above 2^-108.
    bool near;
    __device__ __forceinline__ Weigh(float from_, float c_, float f_) : from(from_), c(c_), f(f_) {
        near = fabsf(from) * c < 0x1p20f && c < 0x1p27f;
        off = -__fmul_rn(from, c);
        if (near) f *= sm100::ex2_approx(-fmaf(from, c, off));  // what the product was rounded by
    }
    __device__ __forceinline__ float2 two(float2 x) const {
        const float2 cc = make_float2(c, c);
        const float2 a = near ? fma_f32x2(x, cc, make_float2(off, off)) : mul_f32x2(add_f32x2(x, make_float2(-from, -from)), cc);
        return mul_f32x2(make_float2(sm100::ex2_approx(a.x), sm100::ex2_approx(a.y)), make_float2(f, f));
    }
    __device__ __forceinline__ float operator()(float x) const { return two(make_float2(x, x)).x; }
    template <typename T>
    __device__ __forceinline__ uint4 vector(uint4 q) const {
        uint32_t* const e = &q.x;
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 y = two(unpack(e[k]));
                e[k] = pack_bf16(y.x, y.y);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
                const float2 y = two(make_float2(__uint_as_float(e[k]), __uint_as_float(e[k + 1])));
                e[k] = __float_as_uint(y.x);
                e[k + 1] = __float_as_uint(y.y);
            }
        }
        return q;
    }
};
// Entries `by` .. of two vectors side by side, 0 < by < kVec; the same `by` in the whole CTA.
template <typename T>
__device__ __forceinline__ uint4 straddle(const uint4& a, const uint4& b, int by) {
    const auto halves = [](uint32_t x, uint32_t y) { return __byte_perm(x, y, 0x5432); };
    if constexpr (sizeof(T) == 4) {
        return by == 1 ? make_uint4(a.y, a.z, a.w, b.x) : by == 2 ? make_uint4(a.z, a.w, b.x, b.y) : make_uint4(a.w, b.x, b.y, b.z);
    } else {
        switch (by) {
            case 1: return make_uint4(halves(a.x, a.y), halves(a.y, a.z), halves(a.z, a.w), halves(a.w, b.x));
            case 2: return make_uint4(a.y, a.z, a.w, b.x);
            case 3: return make_uint4(halves(a.y, a.z), halves(a.z, a.w), halves(a.w, b.x), halves(b.x, b.y));
            case 4: return make_uint4(a.z, a.w, b.x, b.y);
            case 5: return make_uint4(halves(a.z, a.w), halves(a.w, b.x), halves(b.x, b.y), halves(b.y, b.z));
            case 6: return make_uint4(a.w, b.x, b.y, b.z);
            default: return make_uint4(halves(a.w, b.x), halves(b.x, b.y), halves(b.y, b.z), halves(b.z, b.w));
        }
    }
}

template <typename T, int kMode>
__global__ void __launch_bounds__(kThreads, 4)
distill_kernel(const DistillArgs a, int* status) {
    constexpr bool kSums = kMode != kDistillBwd, kGrad = kMode != kDistillLoss;
    constexpr int kVec = Row<T>::kVec;
    cg::cluster_group cluster = cg::this_cluster();
    // a byte for each whole vector of the part: a bit for each of its entries that the teacher names
    extern __shared__ __align__(16) uint8_t held[];
    __shared__ __align__(16) Shared sm;
    const int tid = threadIdx.x, ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int64_t row = blockIdx.x / ctas;
    // this thread's entry
    int id = -1;
    float v = -INFINITY;
    if (tid < a.teacher) {
        id = a.ids[row * a.teacher + tid];
        v = a.values[row * a.teacher + tid];
    }
    const float w = kGrad ? a.weight[row] : 0.f;
    const T* const in = static_cast<const T*>(a.logits) + row * a.stride;
    T* const out = kGrad ? static_cast<T*>(a.grad) + row * a.grad_stride : nullptr;
    const Part<T> part(in, a.vocab, rank, ctas);
    const int whole = part.whole(), last = max(whole - 1, 0) / kBatch * kBatch;  // where the last batch begins
    const uint4* const body = reinterpret_cast<const uint4*>(in + part.body0);
    // The gradient's vectors begin `by` entries into the logits' vectors.
    const int off = kGrad ? (int)((reinterpret_cast<uintptr_t>(out + part.body0) & 15u) / sizeof(T)) : 0;
    const int by = off ? kVec - off : 0;
    // (before it is known whether the row counts: as long as that takes, so does its first batch)
    const uint64_t first_policy = kSums && kGrad ? keep_policy() : drop_policy(), policy = drop_policy();
    uint4 next[kU];
    const auto load_last = [&] {
        if (by)
            load_batch<T, kThreads, true>(next, body, last, whole, policy);
        else
            load_batch<T, kThreads, false>(next, body, last, whole, policy);
    };
    if constexpr (kSums)
        load_batch<T, kThreads, false>(next, body, 0, whole, first_policy);
    else
        load_last();
    if (kSums && tid == 0) fetch<kThreads>(body, 1, kAhead - 1, whole);
    // (whole batches of it, which a thread may read)
    for (int i = tid; i < (whole + kBatch - 1) / kBatch * (kBatch / 16); i += kThreads)
        reinterpret_cast<uint4*>(held)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) sm.edge_held = sm.twice = 0;
    if (id >= a.vocab) {
        if (rank == 0) report_status(status, KDA_ERR_INVALID_ARG);
        id = -1;
    }
    if (id < 0) v = -INFINITY;
    if (tid < a.teacher) sm.ids[tid] = id;
    const auto clear = [&] {  // zeros, by the gradient's own vectors
        const Part<T> zero(out, a.vocab, rank, ctas);
        uint4* const to = reinterpret_cast<uint4*>(out + zero.body0);
        for (int i = tid; i < zero.whole(); i += kThreads) store_vec(to + i, make_uint4(0, 0, 0, 0), policy);
        if (zero.edge(tid) >= 0) out[zero.edge(tid)] = io<T>::from_f(0.f);
    };
    const bool live = __syncthreads_or(id >= 0 && (a.tail || !(v == -INFINITY))) && (kSums || w != 0.f);
    if (!live) {  // the same for the whole cluster
        if (kSums && rank == 0 && tid == 0) {
            a.loss[row] = 0.f;
            if (!kGrad) *reinterpret_cast<float4*>(a.stats + 4 * row) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if constexpr (kGrad) clear();
        return;
    }
    if (kSums && ctas > 1) cluster_arrive();  // other CTAs' shared memory is written below, once all run
    const bool mine = id >= part.e0 && id < part.e1;
    // a part has the logits of its entries, rank 0 of all where there are sums
    // (as it is: nothing waits for it before the sums)
    T raw = io<T>::from_f(0.f);
    if (id >= 0 && (mine || (kSums && rank == 0))) raw = in[id];
    if (mine) {
        const int off = id - part.body0, i = off / kVec;
        const bool edge = id < part.body0 || id >= part.body1;
        const uint32_t bit = 1u << (edge ? (id < part.body0 ? off + kVec : id - part.body1 + kVec) : i % 4 * 8 + off % kVec);
        if (atomicOr(edge ? &sm.edge_held : reinterpret_cast<uint32_t*>(held) + i / 4, bit) & bit) sm.twice = 1;
    }
    // the teacher
    const float s = a.scale, c = s * kLog2e;
    float p, logp, r = 0.f, mass = 1.f;
    if (tid / 32 * 32 < a.teacher) {  // warps with entries
        if (a.tail) {
            p = expf(v);
            int64_t f = id < 0 ? 0 : v <= 8.f ? exp_fixed(v) : 1ll << 52;
            float sum = p;
#pragma unroll
            for (int d = 16; d; d >>= 1) {
                f += __shfl_xor_sync(~0u, f, d);
                sum += __shfl_xor_sync(~0u, sum, d);
            }
            if (tid % 32 == 0) {
                sm.mass[tid / 32] = f;
                sm.given[tid / 32].x = sum;
            }
        } else {
            const float3 q = lane_sums<false>(make_float3(v, v > -INFINITY ? 1.f : 0.f, 0.f), 32, kLog2e);
            if (tid % 32 == 0) sm.given[tid / 32] = make_float2(q.x, q.y);
        }
    } else if (tid % 32 == 0) {
        sm.mass[tid / 32] = 0;
        sm.given[tid / 32] = make_float2(a.tail ? 0.f : -INFINITY, 0.f);
    }
    __syncthreads();
    if (a.tail) {
        logp = v;
        int64_t f = 0;
        float sum = 0.f;
        for (int k = 0; k * 32 < a.teacher; ++k) {
            f += sm.mass[k];
            sum += sm.given[k].x;
        }
        const int64_t left = (1ll << 40) - f;  // what the entries leave
        r = !(sum == sum) ? sum : left > 0 ? (float)left * 0x1p-40f : 0.f;
        mass = left > 0 ? 1.f : sum;
    } else {
        const float2 e = sm.given[tid % kWarps];
        const float3 q = lane_sums<false>(make_float3(e.x, e.y, 0.f), kWarps, kLog2e);
        const float d = v - q.x;
        p = v == -INFINITY ? 0.f : expf(d) / q.y;
        logp = d - logf(q.y);
    }
    const bool twice = sm.twice != 0;
    bool leads = mine;  // the first of the entries with its token
    if (twice && mine)
        for (int k = 0; k < tid; ++k) leads &= sm.ids[k] != id;
    if (tid < a.teacher) sm.p[tid] = p;
    float m, z, mr, zr;
    if constexpr (kSums) {
        // the tokens outside
        Online o;
        const float lim = limit(c);
        if (part.edge(tid) >= 0 && !(sm.edge_held >> tid & 1)) add_one(o, io<T>::to_f(in[part.edge(tid)]), c, lim);
        stream<T, kThreads, false, false, true>(body, whole, first_policy, next, [&](uint4 (&q)[kU], int j) {
            uint32_t h[kU], any = 0;  // (the bytes beyond the part's vectors are there, and no matter)
#pragma unroll
            for (int u = 0; u < kU; ++u) any |= h[u] = held[j + tid + u * kThreads];
            if (any)
#pragma unroll
                for (int u = 0; u < kU; ++u) drop<T>(q[u], h[u]);
            add_vectors<T, false>(o, q, c, lim);
        });
        // Backwards where the gradient follows: what was read last is likeliest to be in L2.
        if constexpr (kGrad) load_last();
        float3 q = warp_sums<false>(o, c, lim);
        if (tid % 32 == 0) sm.outside[tid / 32] = q;
        if (tid / 32 * 32 < a.teacher) {  // and the entries
            const float xi = io<T>::to_f(raw);
            q = lane_sums<false>(make_float3(leads ? xi : -INFINITY, leads && xi > -INFINITY ? 1.f : 0.f, 0.f), 32, c);
            if (tid % 32 == 0) sm.entries[tid / 32] = make_float2(q.x, q.y);
        } else if (tid % 32 == 0) {
            sm.entries[tid / 32] = make_float2(-INFINITY, 0.f);
        }
        __syncthreads();
        q = lane_sums<false>(sm.outside[tid % kWarps], kWarps, c);
        if (fabsf(q.x) >= lim && fabsf(q.x) < INFINITY) {
            __syncthreads();
            q = far_sums<T, kThreads, false>(in, part, held, sm.edge_held, q.x, c);
            if (tid % 32 == 0) sm.outside[tid / 32] = q;
            __syncthreads();
            q = lane_sums<false>(sm.outside[tid % kWarps], kWarps, c);
        }
        const float2 e0 = sm.entries[tid % kWarps];
        float3 e = lane_sums<false>(make_float3(e0.x, e0.y, 0.f), kWarps, c);
        if (ctas > 1) {
            cluster_wait();
            if (tid < ctas) {
                *cluster.map_shared_rank(&sm.sums[rank], tid) = make_float4(q.x, q.y, e.x, e.y);
                if (rank == 0) *cluster.map_shared_rank(&sm.teacher, tid) = make_float2(r, mass);
            }
            cluster_arrive();
            cluster_wait();
            if (!kGrad && rank != 0) return;
            const float4 each = sm.sums[tid % ctas];
            q = lane_sums<false>(make_float3(each.x, each.y, 0.f), ctas, c);
            e = lane_sums<false>(make_float3(each.z, each.w, 0.f), ctas, c);
            r = sm.teacher.x;
            mass = sm.teacher.y;
        }
        mr = q.x;
        zr = q.y;
        m = max_nan(mr, e.x);
        z = zr * sm100::ex2_approx(octaves(mr, m, c)) + e.y * sm100::ex2_approx(octaves(e.x, m, c));
        if (!(m < INFINITY && m > -INFINITY)) z = __int_as_float(0x7fffffff);  // no distribution
        if (rank == 0) {
            float term = id >= 0 && !(p == 0.f) ? p * (logp - scaled(io<T>::to_f(raw), m, s, logf(z))) : 0.f;
#pragma unroll
            for (int d = 16; d; d >>= 1) term += __shfl_xor_sync(~0u, term, d);
            if (tid % 32 == 0) sm.loss[tid / 32] = term;
        }
    } else {
        const float4 q = *reinterpret_cast<const float4*>(a.stats + 4 * row);
        m = q.x;
        z = q.y;
        mr = q.z;
        zr = q.w;
    }
    const float g = w * s, each = g * mass / z;
    if (kGrad && w == 0.f) {  // (whatever the logits are)
        clear();
    } else if constexpr (kGrad) {
        // outside the entries: one factor times exp2((x - m_r) c)
        float f = each * sm100::ex2_approx(octaves(mr, m, c)), from = mr;
        if (a.tail && zr > 0.f) f -= g * r / zr;
        if (mr == -INFINITY) from = 0.f;  // nothing outside has weight
        const int full = by ? whole - 1 : whole;
        uint4* const to = reinterpret_cast<uint4*>(out + part.body0 + by);
        const Weigh weigh(from, c, f);
        if (by == 0) {
            stream<T, kThreads, false, true, false>(body, whole, policy, next, [&](const uint4 (&q)[kU], int j) {
                uint4* const p = to + j + tid;
                if (j + kBatch <= whole) {
#pragma unroll
                    for (int u = 0; u < kU; ++u) store_vec(p + u * kThreads, weigh.template vector<T>(q[u]), policy);
                } else {
#pragma unroll
                    for (int u = 0; u < kU; ++u)
                        if (j + tid + u * kThreads < whole) store_vec(p + u * kThreads, weigh.template vector<T>(q[u]), policy);
                }
            });
        } else {  // a lane's vector and the next lane's; behind the warp's run a vector of the next warp's
            const int lane = tid % 32, first = Mine<kThreads, true>::first();
            stream<T, kThreads, true, true, false>(body, whole, policy, next, [&](const uint4 (&q)[kU], int j) {
                const int behind = j + first + (kU - 1) * 32 + 1;
                uint4 after = make_uint4(0, 0, 0, 0);
                if (lane == 31 && behind < whole) after = load_vec(body + behind, policy);
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const uint4 give = lane == 0 && u + 1 < kU ? q[u + 1 < kU ? u + 1 : u] : q[u];
                    uint4 n;
                    n.x = __shfl_sync(~0u, give.x, (lane + 1) % 32);
                    n.y = __shfl_sync(~0u, give.y, (lane + 1) % 32);
                    n.z = __shfl_sync(~0u, give.z, (lane + 1) % 32);
                    n.w = __shfl_sync(~0u, give.w, (lane + 1) % 32);
                    if (u + 1 == kU && lane == 31) n = after;
                    if (j + first + u * 32 < full)
                        store_vec(to + j + first + u * 32, weigh.template vector<T>(straddle<T>(q[u], n, by)), policy);
                }
            });
        }
        // entries beside the logits' vectors, and those of them beside the gradient's
        int e = part.edge(tid);
        if (by && whole > 0 && tid >= 2 * kVec && tid < 3 * kVec) {
            e = tid - 2 * kVec;  // `by` before the first and kVec - by after the last
            e = e < by ? part.body0 + e : part.body1 - kVec + e;
        }
        if (e >= 0) out[e] = io<T>::from_f(weigh(io<T>::to_f(in[e])));
    }
    __syncthreads();
    if constexpr (kGrad)
        if (leads && w != 0.f) {
            float given = p;
            if (twice) {  // in the entries' order
                given = 0.f;
                for (int k = 0; k < a.teacher; ++k)
                    if (sm.ids[k] == id) given += sm.p[k];
            }
            out[id] = io<T>::from_f(each * sm100::ex2_approx(octaves(io<T>::to_f(raw), m, c)) - g * given);
        }
    if (kSums && rank == 0 && tid == 0) {
        float loss = 0.f;
        for (int k = 0; k * 32 < a.teacher; ++k) loss += sm.loss[k];
        if (a.tail && !(r == 0.f)) loss += r * (logf(r) - (scaled(mr, m, s, -logf(zr)) - logf(z)));
        a.loss[row] = loss;
        if (!kGrad) *reinterpret_cast<float4*>(a.stats + 4 * row) = make_float4(m, z, mr, zr);
    }
}

template <typename T, int kMode>
cudaError_t launch_typed(const DistillArgs& a, int ctas, int* status, cudaStream_t stream) {
    static std::atomic<uint64_t> raised{0};
    cudaError_t e = raise_smem(distill_kernel<T, kMode>, kDistillRow / 16 + kBatch, raised);
    if (e != cudaSuccess) return e;
    const int64_t body = a.vocab / Row<T>::kVec;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.rows * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)((body + ctas - 1) / ctas + kBatch - 1) / kBatch * kBatch;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = ctas > 1;
    return cudaLaunchKernelEx(&cfg, distill_kernel<T, kMode>, a, status);
}
template <typename T>
cudaError_t launch_mode(const DistillArgs& a, DistillMode mode, int ctas, int* status, cudaStream_t stream) {
    switch (mode) {
        case kDistillLoss: return launch_typed<T, kDistillLoss>(a, ctas, status, stream);
        case kDistillBwd: return launch_typed<T, kDistillBwd>(a, ctas, status, stream);
        default: return launch_typed<T, kDistillBoth>(a, ctas, status, stream);
    }
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, DistillMode mode, int* status, cudaStream_t stream) {
    const int64_t bytes = (int64_t)a.vocab * (a.dtype == KDA_BF16 ? 2 : 4);
    int ctas = 1;
    // Few rows are split over a cluster, as long as its CTAs are two to an SM and a thread has a vector: 64 rows of
    // 32,000 bf16 entries take 5.5 us on four CTAs each, 6.7 on eight.  Gradients take parts of at most 128 KB in rows
    // of up to 1 MB (above, eight CTAs with up to 192 KB): the 608 CTAs that run at a time then have 78 MB under way,
    // which L2 keeps for the second pass (4,096 rows of 131,072 bf16 entries: 427 us with one CTA a row, 384 with two,
    // 406 with four), and a last wave is shorter (the gradient alone, 1,300 rows: 114, 106 and 104 us; 304 rows: 28, 23
    // and 26).
    constexpr int64_t kPart = 128 * 1024;
    while (ctas < kDistillCluster && ((a.rows * ctas * 2 <= 2 * kPlanSMs && bytes / (ctas * 2) >= kThreads * 16) ||
                                      (mode != kDistillLoss && bytes > ctas * kPart)))
        ctas *= 2;
    return a.dtype == KDA_BF16 ? launch_mode<__nv_bfloat16>(a, mode, ctas, status, stream)
                               : launch_mode<float>(a, mode, ctas, status, stream);
}

}  // namespace kda
