// kda_paged_append.cu — new keys and values into the pages of an 8-bit cache.
//
// A page holds page_size tokens of one head in e4m3 with one fp32 scale s:  x = code * s.
//     s_new = the smallest power of two >= 2^-100 with max|x| <= 448 s_new over the tokens written
//     s     = max(s_old, s_new) in a page that already holds tokens, s_new in a fresh one
//     code  = x / s to the nearest e4m3, ties to even;   held codes: code * (s_old / s), if s grew
// Powers of two: e4m3 is a floating format, so a scale only places its range, and dividing by a
// power of two is exact.  The codes then do not depend on how a division rounds, and coding held
// tokens again (a shift of the exponent) loses nothing but what falls below the subnormals.
//
// What bounds it: 2 bytes read and 1 written per element, no reuse.  32,768 tokens of 8 heads (201
// MB) take 34.6 us, 87% of the measured copy bandwidth; the first version, 46 us, issued 170
// instructions per 8 elements of a lane, most of them to find the groups.  640 tokens of a decode
// step take 5 us, which is one chain of launch, slots, rows, scale, stores.
//
// A group is the tokens of a call that share a page; a block finds the groups that begin in its
// tokens from the places where the page changes (a bit mask).  A group of up to 8 tokens (decode)
// is one warp's, a longer one (prefill) its block's four warps', and either keeps its rows in
// registers between the maximum and the coding, so the inputs are read once.
#include "kda_common.cuh"
#include "kda_paged.cuh"

namespace kda {
namespace {

constexpr int kAppendWarps = 4;
constexpr int kMaxPage = 128;

__device__ __forceinline__ uint16_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint16_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// Largest |x| of eight bf16 and of what m holds: the even ones' bits below, the odd ones' above
// (an infinity or NaN: >= 0x7f80).
__device__ __forceinline__ uint32_t amax_pair(const uint4& v, uint32_t m) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    return m;
}
// Largest |x| of the finite ones, as bits of a bf16 in the upper half.
__device__ __forceinline__ uint32_t finite_amax_bits(const uint4& v, uint32_t m) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = (w[i] << 16) & 0x7fff0000u, hi = w[i] & 0x7fff0000u;
        m = max(m, max(lo < 0x7f800000u ? lo : 0u, hi < 0x7f800000u ? hi : 0u));
    }
    return m;
}

// Smallest power of two s >= 2^-100 with amax <= 448 s = 1.75 * 2^8 s.
__device__ __forceinline__ float scale_for(float amax) {
    const uint32_t b = __float_as_uint(amax);
    int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);  // biased exponent
    return __uint_as_float((uint32_t)max(e, 27) << 23);                  // 27 - 127 = -100
}

// Eight codes of x / s where every x is finite and s a power of two: x * inv is x / s exactly.
__device__ __forceinline__ uint2 code8(const uint4& v, float inv) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        const float2 y = mul_f32x2(x, make_float2(inv, inv));
        c[i] = to_e4m3x2(y.x, y.y);
    }
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}
// Of any x and s; an infinity becomes NaN, so that it is not taken for 448.
__device__ __noinline__ uint2 code8_any(uint4 v, float s) {
    auto coded = [&](float x) { return fabsf(x) == INFINITY ? NAN : __fdiv_rn(x, s); };
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
    for (int i = 0; i < 4; ++i)
        c[i] = to_e4m3x2(coded(__uint_as_float(w[i] << 16)), coded(__uint_as_float(w[i] & 0xffff0000u)));
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

struct Tensor {
    const __nv_bfloat16* x;  // this head's rows
    int64_t stride;
    uint8_t* cache;
    float* scale;
};

// One group: tokens t .. t + m - 1, all in `page`.  kWarps warps (this one is `warp`), two rows of
// 256 bytes per warp and step, kSteps steps.
template <int kWarps, int kSteps>
__device__ __forceinline__ void append_group(const AppendArgs& a, const Tensor& x, int head,
                                             int64_t t, int m, const int32_t* slots, int page,
                                             int warp, int lane, uint32_t* red) {
    const int half = lane >> 4, col = (lane & 15) * 8;
    const int64_t ph = (int64_t)page * a.kv_heads + head;
    uint8_t* base = x.cache + ph * a.page_size * kDim;
    const int mask = a.page_size - 1, first = slots[0] & mask;
    const float old = x.scale[ph];
    uint4 v[kSteps];
    uint32_t mx = 0;
    const int r0 = warp * 2 + half;
    const __nv_bfloat16* from = x.x + (t + r0) * x.stride + col;
    const int64_t step = kWarps * 2 * x.stride;
#pragma unroll
    for (int i = 0; i < kSteps; ++i, from += step) {
        v[i] = make_uint4(0, 0, 0, 0);
        if (r0 + i * kWarps * 2 < m) v[i] = __ldg(reinterpret_cast<const uint4*>(from));
    }
    auto largest = [&](uint32_t mine) {
        mine = __reduce_max_sync(~0u, mine);
        if (kWarps > 1) {
            __syncthreads();
            if (lane == 0) red[warp] = mine;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mine = max(mine, red[w]);
        }
        return mine;
    };
#pragma unroll
    for (int i = 0; i < kSteps; ++i) mx = amax_pair(v[i], mx);
    mx = largest(max(mx << 16, mx & 0xffff0000u));
    const bool finite = mx < 0x7f800000u;
    if (!finite) {
        mx = 0;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) mx = finite_amax_bits(v[i], mx);
        mx = largest(mx);
    }
    float s = scale_for(__uint_as_float(mx));
    const bool grew = first > 0 && s > old;
    if (first > 0 && !(s > old)) s = old;  // (a NaN stays one: held codes have no value under it)
    const bool plain = finite && (__float_as_uint(s) & 0x7fffffu) == 0;
    const float inv = 1.f / s;
    base += col;
    if (plain) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int r = r0 + i * kWarps * 2;
            if (r < m) *reinterpret_cast<uint2*>(base + (slots[r] & mask) * kDim) = code8(v[i], inv);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int r = r0 + i * kWarps * 2;
            if (r < m) *reinterpret_cast<uint2*>(base + (slots[r] & mask) * kDim) = code8_any(v[i], s);
        }
    }
    base -= col;
    if (grew) {  // the tokens held before, 16 codes a lane
        const float ratio = __fdiv_rn(old, s);
        for (int i = warp * 32 + lane; i < first * (kDim / 16); i += kWarps * 32) {
            uint4* p = reinterpret_cast<uint4*>(base) + i;
            uint4 c = *p;
            uint32_t* w = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 lo = from_e4m3x2((uint16_t)w[j]), hi = from_e4m3x2((uint16_t)(w[j] >> 16));
                w[j] = to_e4m3x2(lo.x * ratio, lo.y * ratio) |
                       (uint32_t)to_e4m3x2(hi.x * ratio, hi.y * ratio) << 16;
            }
            *p = c;
        }
    }
    // every reader of the old scale has it in a register: __syncthreads above, or one warp
    if (warp == 0 && lane == 0) x.scale[ph] = s;
}

// Block: the groups that begin in tokens [blockIdx.x * chunk, + chunk), chunk <= 128, of head
// blockIdx.y, keys or values by blockIdx.z.  kSteps: steps of the longest group (a page);
// kShortRows: the longest group of one warp.
template <int kSteps, int kShortRows>
__global__ void __launch_bounds__(kAppendWarps * 32, kSteps == 16 ? 5 : 8)
paged_append_kernel(const AppendArgs a, int chunk, int* status) {
    constexpr int kWindow = 2 * kMaxPage;  // a group that begins in the chunk ends in the window
    __shared__ uint32_t change[kWindow / 32 + 1];  // tokens whose page is not that of the one before
    __shared__ int32_t slots[kWindow];
    __shared__ int2 longs[kMaxPage / kShortRows];  // (token, tokens) of the whole block's groups
    __shared__ int count;
    __shared__ uint32_t red[kAppendWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, head = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    const int64_t t0 = (int64_t)blockIdx.x * chunk;
    const int shift = 31 - __clz(a.page_size);
    if (tid == 0) {
        count = 0;
        change[kWindow / 32] = ~0u;  // nothing is beyond the window
    }
#pragma unroll
    for (int i = 0; i < kWindow; i += kAppendWarps * 32) {
        const int64_t t = t0 + i + tid;
        const int slot = t < a.total_tokens ? a.slots[t] : -1;
        const int before = t > 0 && t < a.total_tokens ? a.slots[t - 1] : -1;
        slots[i + tid] = slot;
        const bool other = slot < 0 || before < 0 || slot >> shift != before >> shift;
        const uint32_t m = __ballot_sync(~0u, other);
        if (lane == 0) change[(i >> 5) + warp] = m;
    }
    __syncthreads();
    Tensor x;
    x.x = static_cast<const __nv_bfloat16*>(is_v ? a.v : a.k) + head * kDim;
    x.stride = is_v ? a.v_stride : a.k_stride;
    x.cache = is_v ? a.v_cache : a.k_cache;
    x.scale = is_v ? a.v_scale : a.k_scale;
    int nth = 0;  // the chunk's page changes, one warp after the other
    for (int w0 = 0; w0 < chunk; w0 += 32) {
        uint32_t begins = change[w0 >> 5] & (chunk - w0 < 32 ? (1u << (chunk - w0)) - 1 : ~0u);
        for (; begins; begins &= begins - 1, ++nth) {
            if (nth % kAppendWarps != warp) continue;
            const int i = w0 + __ffs(begins) - 1, slot = slots[i];
            if (slot < 0) continue;
            const int page = slot >> shift;
            if (page >= a.num_pages) {
                if (lane == 0) report_status(status, KDA_ERR_INVALID_ARG);
                continue;
            }
            int w = (i + 1) >> 5;  // the next change
            uint32_t bits = change[w] & (~0u << ((i + 1) & 31));
            while (bits == 0) bits = change[++w];
            const int m = min(min(w * 32 + __ffs(bits) - 1, kWindow) - i, a.page_size);
            if (m <= kShortRows)
                append_group<1, kShortRows / 2>(a, x, head, t0 + i, m, slots + i, page, 0, lane, nullptr);
            else if (lane == 0)
                longs[atomicAdd(&count, 1)] = make_int2(i, m);
        }
    }
    __syncthreads();
    const int groups = count;
    for (int i = 0; i < groups; ++i)  // groups differ in their pages: their order does not matter
        append_group<kAppendWarps, kSteps>(a, x, head, t0 + longs[i].x, longs[i].y, slots + longs[i].x,
                                           slots[longs[i].x] >> shift, warp, lane, red);
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs& a, int* status, cudaStream_t stream) {
    // Tokens per block, a power of two (as pages are): about 1,024 blocks until a block has 128.
    // 2,048 tokens (256 requests of 8) of 8 heads in pages of 64 took 8.9 us with 8,192 blocks,
    // 4.7 with 2,048 and 4.1 with 1,024: a block's own cost is finding its groups.
    const int64_t want = a.total_tokens * a.kv_heads * 2 / 1024;
    int chunk = kAppendWarps;
    while (chunk < kMaxPage && 2 * chunk <= want) chunk *= 2;
    const dim3 grid((unsigned)((a.total_tokens + chunk - 1) / chunk), a.kv_heads, 2);
    // Whole pages of 16 are a warp's each where a block has more than two of them (32,768 tokens of 8
    // heads 36 us, 51 with four warps a page); the longer code costs single tokens 3.8 against 3.3 us.
    void (*const kernel)(const AppendArgs, int, int*) =
        a.page_size == 16   ? (chunk >= 32 ? paged_append_kernel<2, 16> : paged_append_kernel<2, 8>)
        : a.page_size == 32 ? paged_append_kernel<4, 8>
        : a.page_size == 64 ? paged_append_kernel<8, 8> : paged_append_kernel<16, 8>;
    kernel<<<grid, kAppendWarps * 32, 0, stream>>>(a, chunk, status);
    return cudaGetLastError();
}

}  // namespace kda
