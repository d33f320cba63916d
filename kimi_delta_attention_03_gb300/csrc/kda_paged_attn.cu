// kda_paged_attn.cu — attention over a paged cache held in e4m3 with a scale per (page, head).
//
// For row (token i of a run of L, query head h) of a request with context c, over keys
// j = 0 .. c - L + i of head h / (H / Hkv):
//     z_j = (q . k_j) s_k(page of j) sm_scale,   o = sum_j e^(z_j - m) v_j s_v / sum_j e^(z_j - m)
// A row that sees no key gives zeros.  One block per (token, query head): a thread per key for the
// scores, a thread per channel for the sum, with a running maximum.
#include "kda_common.cuh"
#include "kda_paged.cuh"

namespace kda {
namespace {

__device__ __forceinline__ float4 from_e4m3x4(uint32_t c) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(c));
    const float2 x = __half22float2(*reinterpret_cast<__half2*>(&lo));
    const float2 y = __half22float2(*reinterpret_cast<__half2*>(&hi));
    return make_float4(x.x, x.y, y.x, y.y);
}

__global__ void __launch_bounds__(kDim) paged_attention_kernel(const AttnArgs a, int* status) {
    __shared__ float q[kDim], p[kDim], red[4];
    __shared__ int64_t rows[kDim];  // cache row (128 bytes) of each key of the tile, -1: none
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t = blockIdx.x;
    const int head = blockIdx.y, kv = head / (a.heads / a.kv_heads);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (t * a.heads + head) * kDim;
    if (t < a.cu[0] || t >= a.cu[a.num_seqs]) {
        out[tid] = __float2bfloat16_rn(0.f);
        return;
    }
    const int n = seq_of_row(a.cu, a.num_seqs, (int)t);
    if (t - a.cu[n] >= a.max_run) {
        report_status(status, KDA_ERR_INVALID_ARG);
        return;
    }
    const int64_t keys = (int64_t)a.context[n] - (a.cu[n + 1] - t) + 1;
    q[tid] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[t * a.q_stride + head * kDim + tid]) *
             a.sm_scale * 1.4426950408889634f;
    float m = -INFINITY, sum = 0.f, o = 0.f;
    for (int64_t j0 = 0; j0 < keys; j0 += kDim) {
        __syncthreads();
        const int64_t j = j0 + tid;
        float z = -INFINITY, vs = 0.f;
        int64_t row = -1;
        if (j < keys) {
            const int64_t b = j / a.page_size;
            const int page = b < a.width ? a.tables[(int64_t)n * a.width + b] : -1;
            if (page < 0 || page >= a.num_pages) {
                report_status(status, KDA_ERR_INVALID_ARG);
            } else {
                const int64_t ph = (int64_t)page * a.kv_heads + kv;
                row = ph * a.page_size + j % a.page_size;
                const uint32_t* k = reinterpret_cast<const uint32_t*>(a.k_cache + row * kDim);
                float d = 0.f;
                for (int c = 0; c < kDim / 4; ++c) {
                    const float4 x = from_e4m3x4(k[c]);
                    d += x.x * q[4 * c] + x.y * q[4 * c + 1] + x.z * q[4 * c + 2] + x.w * q[4 * c + 3];
                }
                z = d * a.k_scale[ph];
                vs = a.v_scale[ph];
            }
        }
        rows[tid] = row;
        float top = z;
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
        if (lane == 0) red[warp] = top;
        __syncthreads();
        top = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
        const float base = top == -INFINITY ? 0.f : top;
        const float e = exp2f(z - base), keep = exp2f(m - base);
        p[tid] = e * vs;
        float part = e;
        for (int d = 16; d; d >>= 1) part += __shfl_xor_sync(~0u, part, d);
        __syncthreads();
        if (lane == 0) red[warp] = part;
        __syncthreads();
        sum = sum * keep + red[0] + red[1] + red[2] + red[3];
        o *= keep;
        m = top;
        for (int i = 0; i < kDim; ++i)
            if (rows[i] >= 0) {
                uint32_t h;
                const uint16_t c = a.v_cache[rows[i] * kDim + tid];
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
                o += p[i] * __low2float(*reinterpret_cast<__half2*>(&h));
            }
    }
    out[tid] = __float2bfloat16_rn(sum > 0.f ? o / sum : 0.f);
}

}  // namespace

size_t paged_attention_workspace(int32_t, int32_t, int32_t) { return 0; }

cudaError_t launch_paged_attention(const AttnArgs& a, int* status, cudaStream_t stream,
                                   uint64_t* launches) {
    if (a.total_tokens == 0) return cudaSuccess;
    paged_attention_kernel<<<dim3((unsigned)a.total_tokens, a.heads), kDim, 0, stream>>>(a, status);
    ++*launches;
    return cudaGetLastError();
}

}  // namespace kda
