// kda_vocab.cuh — operators over rows of vocabulary logits (log probabilities, distillation): their
// launchers, called by kda_api.cu, and the running sums of a softmax that their kernels share.
//
// A row of logits x with scale s has the distribution exp((x_v - m) s) / z, m = max x, z = sum_v
// exp((x_v - m) s).  A thread takes its entries in one pass with a reference of its own, the
// largest entry so far at the time it was last raised: it is raised (and the sums rescaled) only
// where an entry exceeds it by 2^kSlack, which after a thread's first entries is rare, and the sums
// are brought to the row's maximum at the end.  Differences are formed before they are scaled, so
// that entries near the type's lowest value (a common mask) neither overflow nor lose their order.
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
// Running sums of a thread: z of exp2((x - m) c), and (kEntropy) t of exp2((x - m) c) (x - m) c.
struct Online {
    float m = -INFINITY, top = -INFINITY;  // reference, largest entry
    float2 z = {0.f, 0.f}, t = {0.f, 0.f};
};
__device__ __forceinline__ void rise(Online& o, float to, float c) {
    if (to == -INFINITY) return;
    if (!(to < INFINITY)) {  // NaN or +inf: the row has no distribution
        o.z.x = __int_as_float(0x7fffffff);
        o.m = to;
        return;
    }
    const float d = fmaxf((o.m - to) * c, kFloor), f = sm100::ex2_approx(d);
    o.t = make_float2((o.t.x + o.z.x * d) * f, (o.t.y + o.z.y * d) * f);
    o.z = make_float2(o.z.x * f, o.z.y * f);
    o.m = to;
}
template <bool kEntropy>
__device__ __forceinline__ void add_pair(Online& o, float2 x, float2 minus, float2 c) {
    float2 a = mul_f32x2(add_f32x2(x, minus), c);
    if constexpr (kEntropy) a = make_float2(fmaxf(a.x, kFloor), fmaxf(a.y, kFloor));
    const float2 e = make_float2(sm100::ex2_approx(a.x), sm100::ex2_approx(a.y));
    o.z = add_f32x2(o.z, e);
    if constexpr (kEntropy) o.t = fma_f32x2(e, a, o.t);
}
// U vectors of entries.  Returns their maximum.
template <typename T, bool kEntropy, int U>
__device__ __forceinline__ float add_vectors(Online& o, const uint4 (&r)[U], float c) {
    const float top = vec_max<T, U>(r);
    o.top = max_nan(o.top, top);
    if (!((top - o.m) * c <= kSlack)) rise(o, top, c);
    if (top == -INFINITY) return top;
    const float2 minus = make_float2(-o.m, -o.m), cc = make_float2(c, c);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if constexpr (sizeof(T) == 2) {
            add_pair<kEntropy>(o, unpack(r[u].x), minus, cc);
            add_pair<kEntropy>(o, unpack(r[u].y), minus, cc);
            add_pair<kEntropy>(o, unpack(r[u].z), minus, cc);
            add_pair<kEntropy>(o, unpack(r[u].w), minus, cc);
        } else {
            add_pair<kEntropy>(o, make_float2(__uint_as_float(r[u].x), __uint_as_float(r[u].y)), minus, cc);
            add_pair<kEntropy>(o, make_float2(__uint_as_float(r[u].z), __uint_as_float(r[u].w)), minus, cc);
        }
    }
    return top;
}
template <bool kEntropy>
__device__ __forceinline__ void add_one(Online& o, float x, float c) {
    o.top = max_nan(o.top, x);
    if (!((x - o.m) * c <= kSlack)) rise(o, x, c);
    if (x == -INFINITY) return;
    const float a = fmaxf((x - o.m) * c, kFloor), e = sm100::ex2_approx(a);
    o.z.y += e;
    if constexpr (kEntropy) o.t.y += e * a;
}
// What sums with reference m weigh against those with reference `to` >= m, and octaves between them.
__device__ __forceinline__ float octaves(float m, float to, float c) {
    return fmaxf((m - to) * c, kFloor);
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
// This thread's vectors of the batch that begins at vector j of `whole`; -inf beyond them.
template <typename T, int kThreads>
__device__ __forceinline__ void load_batch(uint4 (&r)[kU], const uint4* body, int j, int whole, uint64_t policy) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const int i = j + (int)threadIdx.x + u * kThreads;
        const uint32_t none = Row<T>::kNone;
        r[u] = make_uint4(none, none, none, none);
        if (i < whole) r[u] = load_vec(body + i, policy);
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
// Of a thread, brought to its largest entry (its reference may be some octaves below).
template <bool kEntropy>
__device__ __forceinline__ float3 own_sums(const Online& o, float c) {
    const float d = octaves(o.m, o.top, c), f = sm100::ex2_approx(d), z = o.z.x + o.z.y;
    return make_float3(o.top, z * f, kEntropy ? (o.t.x + o.t.y + z * d) * f : 0.f);
}
// Of a thread, through its warp.
template <bool kEntropy>
__device__ __forceinline__ float3 warp_sums(const Online& o, float c) {
    return lane_sums<kEntropy>(own_sums<kEntropy>(o, c), 32, c);
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
