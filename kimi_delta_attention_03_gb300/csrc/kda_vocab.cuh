// kda_vocab.cuh — operators over rows of vocabulary logits (log probabilities, distillation): their
// launchers, called by kda_api.cu, and the running sums of a softmax that their kernels share.
//
// A row of logits x with scale s has the distribution exp((x_v - m) s) / z, m = max x, z = sum_v
// exp((x_v - m) s).  A thread takes its entries in one pass with a reference of its own, the
// largest entry so far at the time it was last raised: it is raised (and the sums rescaled) only
// where an entry exceeds it by 2^kSlack, which after a thread's first entries is rare, and the sums
// are brought to the row's maximum at the end.
//
// With c = s log2(e) a weight's octaves (x - m) c are formed as fma(x, c, -fl(m c)): one instruction, and
// what m c is rounded by is the same for all weights and taken off with the reference.  Where m c is
// large (near the type's lowest value, a common mask; at extreme scales) they are formed as (x - m) c:
// differences first, so that equal entries stay equal.
//
// Rows are streamed by CTAs of 256 threads, four to an SM: a thread has four 16-byte vectors at hand and the next
// four under way, and L2 is asked for the batch after those.  The log probabilities of 4,096 rows of 131,072 bf16
// entries, one alternative each, take 161 to 163 us so (97% of the measured copy bandwidth), 177 without asking
// ahead, 174 with batches of two vectors on six CTAs, 199 with 512 threads on two (not asking ahead).  Asking
// further ahead is slower (loss and gradient: 384 us, four batches 400, six 447), and so was a ring of bulk copies in
// shared memory (275 us): what is under way beyond the 64 KB an SM that the bandwidth needs only makes every other
// load wait.  Four CTAs also cover what comes before and after a row's stream; warps of their own for that had
// too few issue slots (238 us).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kda_common.cuh"
#include "kda_paged.cuh"
#include "kda_sm100.cuh"

namespace kda {

struct LogprobArgs {
    int64_t rows, stride;       // rows `stride` elements apart
    int32_t vocab, dtype, top_k;
    const void* logits;
    const int32_t* tokens;      // or null
    const float* inv_temperature;  // or null
    float *logprobs, *entropy;
    int32_t* top_ids;
    float* top_logprobs;
};
constexpr int kMaxTop = 128;
cudaError_t launch_token_logprobs(const LogprobArgs& a, int* status, cudaStream_t stream);

enum DistillMode { kDistillLoss = 0, kDistillBwd = 1, kDistillBoth = 2 };
struct DistillArgs {
    int64_t rows, stride, grad_stride;
    int32_t vocab, dtype, teacher, tail;  // teacher: entries of a row
    float scale;
    const void* logits;
    const int32_t* ids;      // [rows][teacher]
    const float* values;
    const float* weight;     // [rows]: gradients of the losses
    float *loss, *stats;     // [rows], [rows][4] (read by the backward pass)
    void* grad;
};
constexpr int kMaxTeacher = 256;
constexpr int kDistillCluster = 8;
constexpr int64_t kDistillRow = 8 * 192 * 1024;  // bytes of a row (a byte for 16 stays in shared memory)
cudaError_t launch_distill(const DistillArgs& a, DistillMode mode, int* status, cudaStream_t stream);

namespace vocab {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;       // octaves that an entry may exceed its thread's reference by
constexpr float kFloor = -16384.f;  // octaves below which a weight is zero (keeps 0 * -inf away)

template <typename T> struct Row;
template <> struct Row<__nv_bfloat16> {
    static constexpr int kVec = 8;  // entries of 16 bytes
    static constexpr uint32_t kNone = 0xff80ff80u;  // -inf in every entry
};
template <> struct Row<float> {
    static constexpr int kVec = 4;
    static constexpr uint32_t kNone = 0xff800000u;
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

template <typename T, int U>
__device__ __forceinline__ float vec_max(const uint4 (&r)[U]) {
    if constexpr (sizeof(T) == 2) {
        uint32_t m = max2_nan(max2_nan(r[0].x, r[0].y), max2_nan(r[0].z, r[0].w));
#pragma unroll
        for (int u = 1; u < U; ++u)
            m = max2_nan(m, max2_nan(max2_nan(r[u].x, r[u].y), max2_nan(r[u].z, r[u].w)));
        const float2 f = unpack(m);
        return max_nan(f.x, f.y);
    } else {
        float m = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u)
            m = max_nan(max_nan(m, max_nan(__uint_as_float(r[u].x), __uint_as_float(r[u].y))),
                        max_nan(__uint_as_float(r[u].z), __uint_as_float(r[u].w)));
        return m;
    }
}

// -inf in the place of the entries whose bits are set.
template <typename T>
__device__ __forceinline__ void drop(uint4& r, uint32_t bits) {
    uint32_t* const w = &r.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2) {
            if (bits >> (2 * i) & 1) w[i] = (w[i] & 0xffff0000u) | 0xff80u;
            if (bits >> (2 * i + 1) & 1) w[i] = (w[i] & 0xffffu) | 0xff800000u;
        } else {
            if (bits >> i & 1) w[i] = 0xff800000u;
        }
    }
}

// How large a row's maximum may be where octaves are formed as fma(x, c, -fl(m c)): m c is then rounded by less
// than an octave.  A thread's own reference may be kWide times as large (less than 2^4 octaves); one beyond is
// below all that weighs in such a row, and what it gathered is dropped.  Entries below -2^100 weigh nothing.
constexpr float kWide = 256.f, kLowest = -0x1p100f;
constexpr uint32_t kLowestPair = 0xf180f180u;  // of bf16
__device__ __forceinline__ float limit(float c) { return c > 0x1p-60f && c < 0x1p27f ? 0x1p20f / c : 0.f; }
// (x - m) s - less where the difference may be beyond fp32 (the type's lowest value below a large one, at a small s): by
// halves, with the same bits wherever those are no subnormal values.
__device__ __forceinline__ float scaled(float x, float m, float s, float less) {
    return 2.f * fmaf(fmaf(x, 0.5f, -0.5f * m), s, -0.5f * less);
}
// Octaves, kFloor where a weight is nothing.
__device__ __forceinline__ float octaves(float m, float to, float c) { return fmaxf(scaled(m, to, c, 0.f), kFloor); }

// Running sums of a thread: z of exp2((x - m) c), and (kEntropy) t of exp2((x - m) c) (x - m) c.
struct Online {
    float m = -INFINITY, top = -INFINITY;  // reference, largest entry
    float off = 0.f;                       // -fl(m c)
    float2 z = {0.f, 0.f}, t = {0.f, 0.f};
};
__device__ __forceinline__ void rise(Online& o, float to, float c, float lim) {
    if (to == -INFINITY) return;
    const float off = -__fmul_rn(to, c);
    float f = 0.f, d = 0.f;
    if (fabsf(o.m) < kWide * lim) {
        d = fmaxf(off - o.off, kFloor);
        f = sm100::ex2_approx(d);
        o.t = make_float2((o.t.x + o.z.x * d) * f, (o.t.y + o.z.y * d) * f);
        o.z = make_float2(o.z.x * f, o.z.y * f);
    } else {
        o.z = o.t = make_float2(0.f, 0.f);
    }
    o.m = to;
    o.off = off;
}
template <bool kEntropy>
__device__ __forceinline__ void add_pair(Online& o, float2 x, float2 c) {
    const float2 a = fma_f32x2(x, c, make_float2(o.off, o.off));
    const float2 e = make_float2(sm100::ex2_approx(a.x), sm100::ex2_approx(a.y));
    o.z = add_f32x2(o.z, e);
    if constexpr (kEntropy) o.t = fma_f32x2(e, a, o.t);
}
// kU vectors of entries.  Returns their maximum.
template <typename T, bool kEntropy, int U>
__device__ __forceinline__ float add_vectors(Online& o, const uint4 (&r)[U], float c, float lim) {
    const float top = vec_max<T, U>(r);
    o.top = max_nan(o.top, top);
    if (!((top - o.m) * c <= kSlack)) rise(o, top, c, lim);
    if (top == -INFINITY) return top;
    const float2 cc = make_float2(c, c);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        uint32_t w[4] = {r[u].x, r[u].y, r[u].z, r[u].w};
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (kEntropy) w[i] = max2_nan(w[i], kLowestPair);  // (0 * -inf stays away)
                add_pair<kEntropy>(o, unpack(w[i]), cc);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                float2 x = make_float2(__uint_as_float(w[i]), __uint_as_float(w[i + 1]));
                if (kEntropy) x = make_float2(fmaxf(x.x, kLowest), fmaxf(x.y, kLowest));
                add_pair<kEntropy>(o, x, cc);
            }
        }
    }
    return top;
}
__device__ __forceinline__ void add_one(Online& o, float x, float c, float lim) {
    o.top = max_nan(o.top, x);
    if (!((x - o.m) * c <= kSlack)) rise(o, x, c, lim);
    if (x == -INFINITY) return;
    const float a = fmaxf(fmaf(x, c, o.off), kFloor), e = sm100::ex2_approx(a);
    o.z.y += e;
    o.t.y += e * a;
}

constexpr int kU = 4;  // vectors of a batch that a thread has

// Read again soon, or not needed any more: what of a row the L2 keeps.
__device__ __forceinline__ uint64_t keep_policy() {
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint64_t drop_policy() {
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint4 load_vec(const uint4* p, uint64_t policy) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0,%1,%2,%3}, [%4], %5;"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p), "l"(policy));
    return v;
}
__device__ __forceinline__ void store_vec(uint4* p, uint4 v, uint64_t policy) {
    asm volatile("st.global.L2::cache_hint.v4.u32 [%0], {%1,%2,%3,%4}, %5;" ::"l"(p), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w), "l"(policy) : "memory");
}
// Where in a batch a thread's vectors are: kStep apart from the first.  kRuns: a warp's are one run, so that most
// of a lane's neighbours are in its warp.
template <int kThreads, bool kRuns>
struct Mine {
    static constexpr int kStep = kRuns ? 32 : kThreads;
    static __device__ __forceinline__ int first() {
        return kRuns ? (int)(threadIdx.x / 32 * (32 * kU) + threadIdx.x % 32) : (int)threadIdx.x;
    }
};
// This thread's vectors of the batch that begins at vector j of `whole`; -inf beyond them.
template <typename T, int kThreads, bool kRuns>
__device__ __forceinline__ void load_batch(uint4 (&r)[kU], const uint4* body, int j, int whole, uint64_t policy) {
    using At = Mine<kThreads, kRuns>;
    const int first = j + At::first();
    const uint4* const p = body + first;
    if (j + kThreads * kU <= whole) {
#pragma unroll
        for (int u = 0; u < kU; ++u) r[u] = load_vec(p + u * At::kStep, policy);
    } else {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const uint32_t none = Row<T>::kNone;
            r[u] = make_uint4(none, none, none, none);
            if (first + u * At::kStep < whole) r[u] = load_vec(p + u * At::kStep, policy);
        }
    }
}
constexpr int kAhead = 2;  // batches that L2 is asked for ahead of the one at hand
// One thread: n batches from the b-th on, into L2.
template <int kThreads>
__device__ __forceinline__ void fetch(const uint4* body, int b, int n, int whole) {
    const int j = b * kThreads * kU, count = min(n * kThreads * kU, whole - j);
    if (count > 0)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(body + j), "r"(count * 16) : "memory");
}
// use(vectors, j) for every batch of a part, loaded a batch ahead: `a` has the first one of the order.
template <typename T, int kThreads, bool kRuns, bool kBackwards, bool kFetch, typename Use>
__device__ __forceinline__ void stream(const uint4* body, int whole, uint64_t policy, uint4 (&a)[kU], Use use) {
    constexpr int kBatch = kThreads * kU, kStep = kBackwards ? -kBatch : kBatch;
    const int last = max(whole - 1, 0) / kBatch * kBatch, end = kBackwards ? 0 : last;
    if (whole == 0) return;
#pragma unroll 1
    for (int j = last - end;; j += kStep) {
        uint4 b[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) b[u] = a[u];
        if (j != end) load_batch<T, kThreads, kRuns>(a, body, j + kStep, whole, policy);
        if (kFetch && threadIdx.x == 0) fetch<kThreads>(body, j / kBatch + kAhead, 1, whole);
        use(b, j);
        if (j == end) break;
    }
}

// All threads of a cluster's CTAs: what was written to shared memory before is seen after.
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sums (m, z, t) about the largest of n (a power of two) lanes' m, the same in these lanes.
template <bool kEntropy>
__device__ __forceinline__ float3 lane_sums(float3 q, int n, float c) {
    float m = q.x;
    for (int d = n / 2; d; d >>= 1) m = max_nan(m, __shfl_xor_sync(~0u, m, d));
    const float d0 = octaves(q.x, m, c), f = sm100::ex2_approx(d0);
    float z = q.y * f, t = kEntropy ? (q.z + q.y * d0) * f : 0.f;
    for (int d = n / 2; d; d >>= 1) {
        z += __shfl_xor_sync(~0u, z, d);
        if constexpr (kEntropy) t += __shfl_xor_sync(~0u, t, d);
    }
    return make_float3(m, z, t);
}
// Of a thread, brought to its largest entry, through its warp.
template <bool kEntropy>
__device__ __forceinline__ float3 warp_sums(const Online& o, float c, float lim) {
    float3 q = make_float3(o.top, 0.f, 0.f);
    if (fabsf(o.top) < kWide * lim) {
        const float at = __fmul_rn(o.top, c);
        const float d = -o.off - at - fmaf(o.top, c, -at);  // also what the product was rounded by
        const float f = sm100::ex2_approx(d), z = o.z.x + o.z.y;
        q.y = z * f;
        if (kEntropy) q.z = (o.t.x + o.t.y + z * d) * f;
    }
    return lane_sums<kEntropy>(q, 32, c);
}
// A warp's sums of a part once more, differences first, where the row's maximum is beyond the limit.  held: null,
// or a byte for each whole vector with a bit for each entry that is left out; edges: those of the entries
// beside them.
template <typename T, int kThreads, bool kEntropy, typename Part>
__device__ __noinline__ float3 far_sums(const T* row, const Part& part, const uint8_t* held, uint32_t edges, float top,
                                        float c) {
    float z = 0.f, t = 0.f;
#pragma unroll 4
    for (int e = part.e0 + (int)threadIdx.x; e < part.e1; e += kThreads) {
        const int at = e - part.body0;
        const bool beside = e < part.body0 || e >= part.body1;
        const uint32_t out = beside ? edges >> (e < part.body0 ? at + Part::kVec : e - part.body1 + Part::kVec)
                                    : held ? held[at / Part::kVec] >> at % Part::kVec : 0;
        const float a = octaves(io<T>::to_f(row[e]), top, c), w = out & 1 ? 0.f : sm100::ex2_approx(a);
        z += w;
        t += w * a;
    }
    return lane_sums<kEntropy>(make_float3(top, z, t), 32, c);
}

// A CTA's part of a row: entries [e0, e1), of which [body0, body1) are whole vectors.  ctas: a power of two.
template <typename T>
struct Part {
    static constexpr int kVec = Row<T>::kVec;
    int e0, e1, body0, body1;
    __device__ __forceinline__ Part(const T* row, int vocab, int rank, int ctas) {
        const int off = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
        const int head = off ? min(kVec - off, vocab) : 0, lg = __ffs(ctas) - 1;
        const uint32_t body = (uint32_t)(vocab - head) / kVec;  // at most 2^28
        body0 = head + (int)(body * rank >> lg) * kVec;
        body1 = head + (int)(body * (rank + 1) >> lg) * kVec;
        e0 = rank == 0 ? 0 : body0;
        e1 = rank == ctas - 1 ? vocab : body1;
    }
    __device__ __forceinline__ int whole() const { return (body1 - body0) / kVec; }
    // entries beside the whole vectors, by a number below 2 kVec; < 0: there is none
    __device__ __forceinline__ int edge(int i) const {
        const int e = i < kVec ? body0 - kVec + i : body1 + i - kVec;
        return e >= e0 && e < e1 && i < 2 * kVec ? e : -1;
    }
};

}  // namespace vocab
}  // namespace kda
