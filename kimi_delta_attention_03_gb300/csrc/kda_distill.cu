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
// A row is read once: the CTAs of a cluster keep its parts in shared memory (bulk copies), take the
// entries' logits out (-inf stays in their place), sum the rest, exchange sums, overwrite the part
// with its gradient, put the entries' gradients in, and store it with bulk copies again.
#include <cooperative_groups.h>

#include "kda_vocab.cuh"

namespace kda {
namespace {

namespace cg = cooperative_groups;
using namespace vocab;

constexpr int kThreads = 256, kWarps = kThreads / 32;
static_assert(kMaxTeacher <= kThreads, "a thread has one entry");
constexpr uint32_t kPiece = 16384;              // bytes of one bulk copy
constexpr long long kWaitLimit = 4000000000LL;  // clock cycles (about 2 s)

struct Shared {
    float logit[kMaxTeacher];        // rank 0: the entries' logits
    float sums[kDistillCluster][4];  // every CTA's m_r, z_r and those of its entries
    int32_t ids[kMaxTeacher];
    float p[kMaxTeacher];
    float red_a[kWarps], red_b[kWarps], red_c[kWarps], red_d[kWarps], red_e[kWarps], red_f[kWarps];
    double red_p[kWarps];
    uint64_t full;
};

__device__ __forceinline__ void bulk_in(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void bulk_out(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
                 "r"(smem_u32(src)), "r"(bytes) : "memory");
}

// A CTA's part of a row: entries [e0, e1), entry e at shared place e - base; whole vectors of the row
// start at vector 1 of the buffer, entries before and after them are around them, and what is left
// of the first and last vector holds -inf.
template <typename T>
struct Part {
    static constexpr int kVec = Row<T>::kVec;
    int e0, e1, base, body0, body1, vecs;
    __device__ __forceinline__ Part(const T* row, int vocab, int rank, int ctas) {
        const Cut c = cut_row(row, vocab);
        const int v0 = (int)(c.body * rank / ctas), v1 = (int)(c.body * (rank + 1) / ctas);
        body0 = c.head + v0 * kVec;
        body1 = c.head + v1 * kVec;
        e0 = rank == 0 ? 0 : body0;
        e1 = rank == ctas - 1 ? vocab : body1;
        base = body0 - kVec;
        vecs = v1 - v0 + 2;
    }
};

// Zeros into a row's gradient.
template <typename T>
__device__ __forceinline__ void clear(T* row, int vocab, int rank, int ctas) {
    const Cut c = cut_row(row, vocab);
    uint4* body = reinterpret_cast<uint4*>(row + c.head);
    const int64_t v1 = c.body * (rank + 1) / ctas;
    for (int64_t i = c.body * rank / ctas + threadIdx.x; i < v1; i += kThreads) body[i] = make_uint4(0, 0, 0, 0);
    if (rank == 0 && (int)threadIdx.x < c.head + c.tail)
        row[(int)threadIdx.x < c.head ? threadIdx.x : vocab - c.head - c.tail + threadIdx.x] = io<T>::from_f(0.f);
}

template <typename T>
__device__ __forceinline__ uint32_t scaled_pair(float2 x, float2 minus, float2 c, float f) {
    const float2 a = mul_f32x2(add_f32x2(x, minus), c);
    return pack_bf16(sm100::ex2_approx(a.x) * f, sm100::ex2_approx(a.y) * f);
}

template <typename T, int kMode>
__global__ void __launch_bounds__(kThreads) distill_kernel(const DistillArgs a, int* status) {
    constexpr bool kSums = kMode != kDistillBwd, kGrad = kMode != kDistillLoss;
    constexpr int kVec = Row<T>::kVec;
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ __align__(128) unsigned char dynamic[];
    __shared__ Shared sm;
    T* const x = reinterpret_cast<T*>(dynamic);
    const int tid = threadIdx.x, ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int64_t row = blockIdx.x / ctas;
    const T* in = static_cast<const T*>(a.logits) + row * a.stride;
    T* out = kGrad ? static_cast<T*>(a.grad) + row * a.grad_stride : nullptr;
    // this thread's entry
    int id = -1;
    float v = -INFINITY;
    if (tid < a.teacher) {
        id = a.ids[row * a.teacher + tid];
        if (id >= a.vocab) {
            if (rank == 0) report_status(status, KDA_ERR_INVALID_ARG);
            id = -1;
        }
        if (id >= 0) v = a.values[row * a.teacher + tid];
    }
    const float w = kGrad ? a.weight[row] : 0.f;
    const bool live = __syncthreads_or(id >= 0 && (a.tail || !(v == -INFINITY))) && (kSums || w != 0.f);
    if (!live) {  // the same for the whole cluster
        if (kSums && rank == 0 && tid == 0) {
            a.loss[row] = 0.f;
            if (!kGrad) *reinterpret_cast<float4*>(a.stats + 4 * row) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if constexpr (kGrad) clear(out, a.vocab, rank, ctas);
        return;
    }
    // the row's part
    const Part<T> part(in, a.vocab, rank, ctas);
    const uint32_t bytes = (uint32_t)(part.body1 - part.body0) * sizeof(T);
    if (tid == 0) {
        sm100::mbar_init(&sm.full, 1);
        sm100::mbar_init_fence();
        sm100::mbar_arrive_expect_tx(&sm.full, bytes);
        for (uint32_t at = 0; at < bytes; at += kPiece)
            bulk_in(x + kVec + at / sizeof(T), in + part.body0 + at / sizeof(T), min(kPiece, bytes - at), &sm.full);
    }
    if constexpr (kSums) cluster_arrive();  // other CTAs' shared memory is written below, once all run
    if (tid < 2 * kVec) {  // the first and the last vector
        const int place = tid < kVec ? tid : (part.vecs - 2) * kVec + tid, e = part.base + place;
        if (e >= part.e0 && e < part.e1)
            x[place] = in[e];
        else
            x[place] = io<T>::from_f(-INFINITY);
    }
    // the teacher
    float p, logp, r = 0.f, mass = 1.f;
    if (a.tail) {
        logp = v;
        p = tid < a.teacher ? expf(v) : 0.f;
        // what they leave is a small difference: in 64 bits
        const double sum = block_sum<kWarps>(tid < a.teacher ? exp((double)v) : 0.0, sm.red_p);
        const double left = 1.0 - sum;
        r = left > 0.0 || !(left == left) ? (float)left : 0.f;
        mass = (float)sum + r;
    } else {
        const float top = block_max<kWarps>(v, sm.red_a);
        const float e = v == -INFINITY ? 0.f : expf(v - top);
        const float sum = block_sum<kWarps>(e, sm.red_b);
        p = e / sum;
        logp = v - top - logf(sum);
    }
    const float s = a.scale, c = s * kLog2e;
    if (tid < a.teacher) {
        sm.ids[tid] = id;
        sm.p[tid] = p;
    }
    __syncthreads();  // the barrier is there, the edges are written
    if (!sm100::mbar_wait(&sm.full, 0, kWaitLimit)) report_status(status, kStatusTimeout);
    // take the entries out; of several with one token the one whose number stays there leads
    const bool mine = id >= part.e0 && id < part.e1;
    T* const spot = x + (mine ? id - part.base : 0);
    const float xi = mine ? io<T>::to_f(*spot) : 0.f;
    __syncthreads();
    if (mine) {
        if constexpr (sizeof(T) == 2)
            *reinterpret_cast<uint16_t*>(spot) = (uint16_t)tid;
        else
            *reinterpret_cast<uint32_t*>(spot) = (uint32_t)tid;
    }
    __syncthreads();
    bool leads = false;
    if (mine) {
        if constexpr (sizeof(T) == 2)
            leads = *reinterpret_cast<uint16_t*>(spot) == tid;
        else
            leads = *reinterpret_cast<uint32_t*>(spot) == (uint32_t)tid;
    }
    const bool twice = __syncthreads_or(mine && !leads);
    if (mine) *spot = io<T>::from_f(-INFINITY);
    __syncthreads();
    float m, z, mr, zr;
    if constexpr (kSums) {
        // the tokens outside
        Online o;
        uint4* const vec = reinterpret_cast<uint4*>(dynamic);
        constexpr int kU = 2;
        int i = tid;
        for (; i + kThreads < part.vecs; i += kU * kThreads) {
            const uint4 q[kU] = {vec[i], vec[i + kThreads]};
            add_vectors<T, false>(o, q, c);
        }
        if (i < part.vecs) {
            const uint4 q[1] = {vec[i]};
            add_vectors<T, false>(o, q, c);
        }
        const float top = block_max<kWarps>(o.top, sm.red_c);
        const float sum = block_sum<kWarps>((o.z.x + o.z.y) * sm100::ex2_approx(octaves(o.m, top, c)), sm.red_d);
        // the entries
        const float ltop = block_max<kWarps>(leads ? xi : -INFINITY, sm.red_e);
        const float lsum = block_sum<kWarps>(
            leads && xi > -INFINITY ? sm100::ex2_approx(octaves(xi, ltop, c)) : 0.f, sm.red_f);
        cluster_wait();
        if (tid < ctas)
            *reinterpret_cast<float4*>(cluster.map_shared_rank(&sm.sums[rank][0], tid)) = make_float4(top, sum, ltop, lsum);
        if (mine) *cluster.map_shared_rank(&sm.logit[tid], 0) = xi;
        cluster_arrive();
        cluster_wait();
        m = mr = -INFINITY;
        for (int k = 0; k < ctas; ++k) {
            mr = max_nan(mr, sm.sums[k][0]);
            m = max_nan(m, sm.sums[k][2]);
        }
        m = max_nan(m, mr);
        z = zr = 0.f;
        for (int k = 0; k < ctas; ++k) {
            zr += sm.sums[k][1] * sm100::ex2_approx(octaves(sm.sums[k][0], mr, c));
            z += sm.sums[k][3] * sm100::ex2_approx(octaves(sm.sums[k][2], m, c));
        }
        z += zr * sm100::ex2_approx(octaves(mr, m, c));
        if (!(m < INFINITY && m > -INFINITY)) z = __int_as_float(0x7fffffff);  // no distribution
        if (rank == 0) {
            const float ln_z = logf(z);
            float part_loss = 0.f;
            if (id >= 0 && !(p == 0.f)) part_loss = p * (logp - ((sm.logit[tid] - m) * s - ln_z));
            float loss = block_sum<kWarps>(part_loss, sm.red_a);
            if (tid == 0) {
                if (a.tail && !(r == 0.f)) loss += r * (logf(r) - ((mr - m) * s + logf(zr) - ln_z));
                a.loss[row] = loss;
                if (!kGrad) *reinterpret_cast<float4*>(a.stats + 4 * row) = make_float4(m, z, mr, zr);
            }
        }
    } else {
        const float4 q = *reinterpret_cast<const float4*>(a.stats + 4 * row);
        m = q.x;
        z = q.y;
        mr = q.z;
        zr = q.w;
    }
    if constexpr (kGrad) {
        const float g = w * s, each = g * mass / z;
        // outside the entries: one factor times exp2((x - m_r) c)
        float f = each * sm100::ex2_approx(octaves(mr, m, c)), from = mr;
        if (a.tail && zr > 0.f) f -= g * r / zr;
        if (mr == -INFINITY) from = 0.f;  // nothing outside has weight
        const float2 minus = make_float2(-from, -from), cc = make_float2(c, c);
        uint4* const vec = reinterpret_cast<uint4*>(dynamic);
        for (int i = tid; i < part.vecs; i += kThreads) {
            uint4 q = vec[i];
            uint32_t* const e = &q.x;
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int k = 0; k < 4; ++k) e[k] = scaled_pair<T>(unpack(e[k]), minus, cc, f);
            } else {
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    const float2 y = mul_f32x2(
                        add_f32x2(make_float2(__uint_as_float(e[k]), __uint_as_float(e[k + 1])), minus), cc);
                    e[k] = __float_as_uint(sm100::ex2_approx(y.x) * f);
                    e[k + 1] = __float_as_uint(sm100::ex2_approx(y.y) * f);
                }
            }
            vec[i] = q;
        }
        __syncthreads();
        if (leads) {
            float mass_here = p;
            if (twice) {  // in the entries' order
                mass_here = 0.f;
                for (int k = 0; k < a.teacher; ++k)
                    if (sm.ids[k] == id) mass_here += sm.p[k];
            }
            *spot = io<T>::from_f(each * sm100::ex2_approx((xi - m) * c) - g * mass_here);
        }
        sm100::fence_async_shared();
        __syncthreads();
        if (((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(in)) & 15u) == 0) {
            if (tid == 0) {
                for (uint32_t at = 0; at < bytes; at += kPiece)
                    bulk_out(out + part.body0 + at / sizeof(T), x + kVec + at / sizeof(T), min(kPiece, bytes - at));
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
            if (tid < 2 * kVec) {
                const int place = tid < kVec ? tid : (part.vecs - 2) * kVec + tid, e = part.base + place;
                if (e >= part.e0 && e < part.e1) out[e] = x[place];
            }
            if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        } else {
            for (int e = part.e0 + tid; e < part.e1; e += kThreads) out[e] = x[e - part.base];
        }
    }
}

template <typename T, int kMode>
cudaError_t launch_typed(const DistillArgs& a, int ctas, int* status, cudaStream_t stream) {
    static std::atomic<uint64_t> raised{0};
    const size_t most = kDistillPart + 32;
    cudaError_t e = raise_smem(distill_kernel<T, kMode>, most, raised);
    if (e != cudaSuccess) return e;
    const int64_t body = a.vocab / Row<T>::kVec;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.rows * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)((body + ctas - 1) / ctas + 2) * 16;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
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
    while (ctas < kDistillCluster && (bytes > (int64_t)ctas * 68 * 1024 ||
                                      (a.rows * ctas * 2 <= 2 * kPlanSMs && bytes / (ctas * 2) >= 8192)))
        ctas *= 2;
    return a.dtype == KDA_BF16 ? launch_mode<__nv_bfloat16>(a, mode, ctas, status, stream)
                               : launch_mode<float>(a, mode, ctas, status, stream);
}

}  // namespace kda
