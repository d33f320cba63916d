// kda_paged_attn.cu — attention over a paged cache held in e4m3 with a scale per (page, head).
//
// For row (token i of a run of L, query head h) of a request with context c, over keys
// j = 0 .. c - L + i of key head h / G (G = H / Hkv query heads share one):
//     z_j = (q . k_j) s_k(page of j) sm_scale,   o = sum_j e^(z_j - m) v_j s_v / sum_j e^(z_j - m)
//
// The cache's bytes go from HBM to the tensor cores as they are: both products take the e4m3 tiles
// that TMA puts into shared memory as tcgen05 operands (kind::f8f6f4), 128 keys at a time, so no
// key or value is ever converted.  What meets them is split into e4m3 terms:
//   S^T [128 keys x 2R] = K [128 x 128] [Q_hi; Q_lo]^T    q = (Q_hi + Q_lo / 16) / s: a bf16 has 8
//                        significant bits, two signed 4-bit ones hold them all
//   O^T [128 channels x 3R] += V^T [128 x 128] [P_0 P_1 P_2]    p = P_0 + P_1 + P_2 / 2^9: 11 bits
//                        down to 2^-16 of a row's largest weight, within 2^-25 of it below
// R (8, 16, 32 or 64) rows of one key head are a tile's columns, so one decode token costs an
// eighth of eight, and the terms are extra columns, not extra passes over K and V.
// The page scales never touch a tile either: s_k multiplies the scores of its keys, and log2 s_v is
// added to them, so that p' = p s_v goes into the second product and p' / s_v into the sum.
//
// Work: all (request, key head, row tile, 128-key tile) quadruples in a row, cut into equal shares,
// one per resident CTA, whatever the lengths.  A share's ends inside a (request, head, row tile)
// unit leave partial results (O, m, sum) in the workspace, which a second kernel joins in key
// order; a cut within two tiles of a unit's end, or in a unit of up to four, moves to the end.
//
// Roles of a CTA's warps:
//   softmax warpgroups, one per 16 rows: scores -> weights, one thread per key of the tile (its TMEM
//        lane), and the outputs, one thread per channel.  Row maxima are not taken per tile: weights
//        are formed against a reference that a row's scores may exceed by up to 2^2.5 before the
//        four warps agree (one barrier with a vote) to raise it and rescale their columns of O^T,
//        which after the first tile is rare.
//   producer: work list, page tables and scales a tile ahead, TMA of K, V and raw q
//   issuer of the MMAs: scores of tile j + 1 before the weighted sum of tile j
//
// Masked places.  Keys beyond a row's limit get weight 0.  Values beyond the request's context are
// zeroed in shared memory (0 * NaN), and a NaN value inside it is replaced by 0 in tiles where some
// row may not see it and put back into the rows that do.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "kda_common.cuh"
#include "kda_paged.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int kTileKeys = 128;
constexpr int kTileBytes = kTileKeys * kDim;  // one K or V tile, e4m3
constexpr int kSegs = 4, kMetas = 4;          // work descriptors, tiles' page scales in flight
constexpr int kMaxTilePages = 8;              // pages of 16 tokens in a tile
constexpr int kSnapUnit = 4, kSnapEdge = 2;   // units this short, and cuts this near, are not cut
constexpr int kGrainTiles = 4;                // least share of a CTA
constexpr long long kAttnWaitLimit = 4000000000LL;  // clock cycles (about 2 s)
constexpr float kNoRef = -1e37f;              // reference of a row that has seen no key
constexpr float kLog2e = 1.4426950408889634f;

template <int R>
struct Cfg {
    static constexpr bool kHalf = R >= 32;                  // weights and values meet in f16
    static constexpr int kRW = R == 64 ? 32 : R == 8 ? 8 : 16;  // rows of a softmax warpgroup
    static constexpr int kGroups = R / kRW;                 // softmax warpgroups
    static constexpr int kSoft = kGroups * 128;             // their threads
    static constexpr int kConv = kHalf ? 128 : 0;           // threads that convert values
    static constexpr int kThreads = kSoft + kConv + 64;     // and the producer's and the issuer's
    static constexpr int kTerms = kHalf ? 1 : 3;            // numbers a weight is held in
    static constexpr int kNQ = 2 * R;                       // columns of a score tile
    static constexpr int kNP = (kTerms * R + 15) / 16 * 16; // columns of the output tile
    static constexpr int kCtasPerSm = R <= 16 ? 2 : 1;
    static constexpr int kKStages = R <= 16 ? 2 : 3;
    static constexpr int kVStages = R == 32 ? 3 : 2;
    static constexpr int kTmem = R == 8 ? 64 : R == 16 ? 128 : R == 32 ? 256 : 512;
    static constexpr int kPBytes = 16384;                   // 128 keys x 128 bytes
    static constexpr int kValBytes = kHalf ? 2 * kTileBytes : 0;  // a tile of values in f16
    // weights are 2^kPeak at their row's reference and may reach 2^(kPeak + kSlack), below the
    // format's largest (448 and 65504)
    static constexpr float kPeak = kHalf ? 10.f : 6.f, kSlack = kHalf ? 5.5f : 2.5f;
    static constexpr uint32_t kOffK = 0;
    static constexpr uint32_t kOffV = kOffK + kKStages * kTileBytes;
    static constexpr uint32_t kOffVal = kOffV + kVStages * kTileBytes;
    static constexpr uint32_t kOffP = kOffVal + 2 * kValBytes;
    static constexpr uint32_t kOffQ = kOffP + 2 * kPBytes;
    static constexpr uint32_t kOffRaw = kOffQ + kNQ * 128;
    static constexpr uint32_t kOffSmall = kOffRaw + R * 256;
    static_assert(2 * kNQ + kNP <= kTmem, "tensor memory columns");
    static_assert(kTerms * R * (kHalf ? 2 : 1) <= 128, "a key's weights fill at most a row");
};

// One share of a unit, as the producer hands it to the other warps.
struct Seg {
    int32_t n;             // request; -1: no more work
    int32_t q0;            // first packed row of its run
    int32_t head;          // key head
    int32_t row0, rows;    // rows of the unit in the run's (token, head in group) order
    int32_t tile0, tile1;  // 128-key tiles
    int32_t keys;          // keys the unit's last row sees
    int32_t lim0;          // token i sees keys below lim0 + i
    int32_t slot;          // workspace slot of its partial result, -1: it is the whole unit
    int32_t pad[2];
};

template <int R>
struct Small {
    float mref[R];
    float fac[R];
    int32_t lim[2][R];
    int32_t orow[2][R];
    float red[4][R];
    int32_t first_nan[kSegs][kDim];
    float2 meta[kMetas][kMaxTilePages];
    Seg segs[kSegs];
    uint64_t k_full[Cfg<R>::kKStages], k_empty[Cfg<R>::kKStages];
    uint64_t v_full[Cfg<R>::kVStages], v_empty[Cfg<R>::kVStages];
    uint64_t meta_full[kMetas], meta_empty[kMetas], val_full[2];
    uint64_t seg_full[kSegs], seg_empty[kSegs];
    uint64_t s_full[2], p_ready[2], pv_done[2], raw_full, raw_empty, q_ready;
    uint32_t qred[Cfg<R>::kSoft / 32];
    uint32_t tmem;
    int32_t abort_flag;
    // the share: first unit and tile, and how many tiles
    int64_t scan[Cfg<R>::kThreads / 32];
    int32_t at[2][4];      // (request, head, row tile, tile) of both ends
    int64_t pos[2];
};

template <int R>
constexpr size_t smem_bytes() { return Cfg<R>::kOffSmall + sizeof(Small<R>) + 1024; }
static_assert(smem_bytes<64>() <= 232448 && smem_bytes<32>() <= 232448, "shared memory of a CTA");
static_assert(smem_bytes<16>() <= 115712 && smem_bytes<8>() <= 115712, "shared memory of two CTAs");

// Workspace: per CTA two partial results (the unit it begins in, the unit it ends in).
struct PartDesc {
    int32_t valid, n, head, rt;
    int32_t ends, pad[3];
};
template <int R>
struct Part {
    float o[R][kDim];
    float m[R], l[R];
};

// ------------------------------------------------------------------------------ small wrappers
struct Waiter {
    volatile int32_t* flag;
    int* status;
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
        return mbar_try_wait(bar, parity) || slow(bar, parity);
    }
    __device__ __noinline__ bool slow(uint64_t* bar, uint32_t parity) const {
        const long long t0 = clock64();
        while (!mbar_try_wait_hint(bar, parity, 20000)) {
            if (*flag) return false;
            if (clock64() - t0 > kAttnWaitLimit) {
                *flag = 1;
                report_status(status, kStatusTimeout);
                return false;
            }
        }
        return true;
    }
};

__device__ __forceinline__ void group_sync(int group) {  // the four warps of a warpgroup
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + 2 * group) : "memory");
}
__device__ __forceinline__ bool group_any(int group, bool x) {  // does any of its threads say so
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"((uint32_t)x), "r"(2 + 2 * group) : "memory");
    return r != 0;
}
template <int kCount>
__device__ __forceinline__ bool all_any(bool x) {  // all softmax warpgroups
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 15, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"((uint32_t)x), "n"(kCount) : "memory");
    return r != 0;
}
__device__ __forceinline__ bool conv_any(bool x) {  // the warps that convert values
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 14, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"((uint32_t)x) : "memory");
    return r != 0;
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            saddr(dst)), "l"(src), "r"(bytes), "r"(saddr(bar)) : "memory");
}
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
// Instruction descriptor with both operands' format code 0 (e4m3 for kind::f8f6f4, f16 for
// kind::f16) and fp32 sums, M = 128.
__host__ __device__ constexpr uint32_t idesc_zero(int N, bool a_mn_major, bool b_mn_major) {
    return (1u << 4) | ((uint32_t)a_mn_major << 15) | ((uint32_t)b_mn_major << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// kN (8 or 16) columns of 32-bit values, without a wait: the registers hold them after
// tmem_ld_wait(), which also keeps the compiler from reading them earlier.
template <int kN>
__device__ __forceinline__ void tmem_ld_start(uint32_t addr, float (&r)[kN]) {
    if constexpr (kN == 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]),
                       "=f"(r[6]), "=f"(r[7])
                     : "r"(addr) : "memory");
    else
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
            "%14,%15}, [%16];"
            : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
              "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]),
              "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
            : "r"(addr) : "memory");
}
template <int kN, int kM>
__device__ __forceinline__ void tmem_ld_wait(float (&r)[kM][kN]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int i = 0; i < kN; ++i) asm volatile("" : "+f"(r[m][i]));
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const float (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
                 "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
                 : "memory");
}
__device__ __forceinline__ uint16_t half2_to_e4m3(uint32_t h) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(h));
    return c;
}
__device__ __forceinline__ uint32_t e4m3_to_half2(uint16_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    return h;
}
__device__ __forceinline__ uint16_t float2_to_e4m3(float lo, float hi) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
    return c;
}
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Order-preserving map of floats to integers (for an integer maximum over a warp).
__device__ __forceinline__ int32_t ordered(float x) {
    const int32_t i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int32_t i) {
    return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}

// A key's 16 values of a tile in which some row does not see every key: zeros beyond the context;
// a NaN is replaced by 0 and its first position noted, for the rows that do see it.
__device__ __forceinline__ bool mask_values(uint4& v, bool in, int pos, int32_t* first_nan) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
    if (!in) {
        v = make_uint4(0, 0, 0, 0);
        return true;
    }
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t nan = __vcmpeq4(w[i] & 0x7f7f7f7fu, 0x7f7f7f7fu);
        if (nan) {
            any = true;
            for (int y = 0; y < 4; ++y)
                if (nan >> (8 * y) & 1) atomicMin(first_nan + i * 4 + y, pos);
            w[i] &= ~nan;
        }
    }
    return any;
}

// Sums over the warp of kN values per lane: lane l gets the sum of value l % kN.
template <int kN>
__device__ __forceinline__ float warp_sums(float (&v)[kN], int lane) {
#pragma unroll
    for (int off = kN / 2; off >= 1; off >>= 1) {
        const bool up = lane & off;
#pragma unroll
        for (int i = 0; i < off; ++i) {
            const float keep = up ? v[i + off] : v[i], send = up ? v[i] : v[i + off];
            v[i] = keep + __shfl_xor_sync(~0u, send, off);
        }
    }
#pragma unroll
    for (int off = kN; off < 32; off <<= 1) v[0] += __shfl_xor_sync(~0u, v[0], off);
    return v[0];
}

// ------------------------------------------------------------------------------------ the work
struct Run {
    int32_t q0, len, ctx;
};
__device__ __forceinline__ Run load_run(const AttnArgs& a, int n, int* status) {
    Run r;
    r.q0 = a.cu[n];
    r.len = a.cu[n + 1] - r.q0;
    r.ctx = a.context[n];
    const int cap = a.width * a.page_size;
    if (r.q0 < 0 || r.len < 0 || (int64_t)r.q0 + r.len > a.total_tokens || r.len > a.max_run ||
        r.ctx > cap) {
        if (status) report_status(status, KDA_ERR_INVALID_ARG);
        if (r.q0 < 0 || r.len < 0 || (int64_t)r.q0 + r.len > a.total_tokens) r.len = 0;
        r.ctx = min(r.ctx, cap);
    }
    r.ctx = max(r.ctx, 0);
    return r;
}
// Keys that the last row of row tile rt sees, and the tiles they take (at least one: an empty unit
// has its zeros to write).
template <int R>
__device__ __forceinline__ int unit_keys(const Run& r, int group, int rt) {
    const int last = (min((rt + 1) * R, r.len * group) - 1) / group;
    return max(r.ctx - r.len + 1 + last, 0);
}
template <int R>
__device__ __forceinline__ int unit_tiles(const Run& r, int group, int rt) {
    return max((unit_keys<R>(r, group, rt) + kTileKeys - 1) / kTileKeys, 1);
}
template <int R>
__device__ __forceinline__ int row_tiles(const Run& r, int group) {
    return (r.len * group + R - 1) / R;
}
template <int R>
__device__ __forceinline__ int64_t head_tiles(const Run& r, int group) {
    int64_t s = 0;
    const int nrt = row_tiles<R>(r, group);
    for (int rt = 0; rt < nrt; ++rt) s += unit_tiles<R>(r, group, rt);
    return s;
}

// Turns a cut at tile x of the request that begins at `base` into (request, head, row tile, tile),
// moved to the unit's end where the cut would leave little on one side.
template <int R>
__device__ __forceinline__ void place_cut(const AttnArgs& a, const Run& r, int n, int64_t base,
                                          int64_t per_head, int64_t x, int32_t* at, int64_t* pos) {
    const int group = a.heads / a.kv_heads, nrt = row_tiles<R>(r, group);
    int64_t off = x - base;
    int h = (int)(off / per_head), rt = 0;
    off -= h * per_head;
    int u = unit_tiles<R>(r, group, 0);
    while (off >= u) {
        off -= u;
        u = unit_tiles<R>(r, group, ++rt);
    }
    int t = (int)off;
    int64_t moved = x;
    if (t > 0) {
        const bool down = u <= kSnapUnit ? 2 * t < u : t < kSnapEdge;
        const bool up = u <= kSnapUnit ? !down : u - t < kSnapEdge;
        if (down) {
            moved -= t;
            t = 0;
        } else if (up) {
            moved += u - t;
            t = 0;
            if (++rt == nrt) {
                rt = 0;
                if (++h == a.kv_heads) {
                    h = 0;
                    ++n;  // requests without rows are skipped when the share is walked
                }
            }
        }
    }
    at[0] = n;
    at[1] = h;
    at[2] = rt;
    at[3] = t;
    *pos = moved;
}

// All threads: this CTA's share into sm.at / sm.pos.
template <int R>
__device__ __forceinline__ void find_share(const AttnArgs& a, Small<R>& sm, int* status) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, N = a.num_seqs;
    const int group = a.heads / a.kv_heads;
    constexpr int kThreads = Cfg<R>::kThreads;
    const int per = (N + kThreads - 1) / kThreads, n0 = min(tid * per, N), n1 = min(n0 + per, N);
    int64_t mine = 0;
    for (int n = n0; n < n1; ++n) {
        const Run r = load_run(a, n, blockIdx.x == 0 ? status : nullptr);
        mine += head_tiles<R>(r, group) * a.kv_heads;
    }
    int64_t in = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(~0u, in, d);
        if (lane >= d) in += y;
    }
    if (lane == 31) sm.scan[warp] = in;
    if (tid < 2) sm.pos[tid] = -1;
    __syncthreads();
    int64_t base = in - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) base += sm.scan[w];
        total += sm.scan[w];
    }
    const int64_t ctas = min((int64_t)gridDim.x, max((total + kGrainTiles - 1) / kGrainTiles, (int64_t)1));
    const int64_t c = blockIdx.x;
    for (int e = 0; e < 2; ++e) {
        const int64_t x = c >= ctas ? total : (c + e) * total / ctas;
        if (x >= total) {
            if (tid == 0) {
                sm.pos[e] = total;
                sm.at[e][0] = N;
                sm.at[e][3] = 0;
            }
        } else if (mine > 0 && x >= base && x < base + mine) {
            int64_t b = base;
            for (int n = n0; n < n1; ++n) {
                const Run r = load_run(a, n, nullptr);
                const int64_t ph = head_tiles<R>(r, group);
                if (x < b + ph * a.kv_heads) {
                    place_cut<R>(a, r, n, b, ph, x, sm.at[e], &sm.pos[e]);
                    break;
                }
                b += ph * a.kv_heads;
            }
        }
    }
    __syncthreads();
}

// ---------------------------------------------------------------------------------- the kernel
template <int R>
__global__ void __launch_bounds__(Cfg<R>::kThreads, Cfg<R>::kCtasPerSm)
paged_attention_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap k_map,
                       const __grid_constant__ CUtensorMap v_map, int* status) {
    using C = Cfg<R>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    Small<R>& sm = *reinterpret_cast<Small<R>*>(smem + C::kOffSmall);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kProducer = (C::kSoft + C::kConv) / 32, kIssuer = kProducer + 1;
    const int group = a.heads / a.kv_heads, bs = a.page_size;
    PartDesc* descs = static_cast<PartDesc*>(a.workspace);
    Part<R>* parts = reinterpret_cast<Part<R>*>(static_cast<char*>(a.workspace) +
                                                (size_t)gridDim.x * 2 * sizeof(PartDesc));

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    find_share<R>(a, sm, status);
    if (tid < 2) {  // partial results of this CTA: none so far
        PartDesc d = {};
        descs[2 * blockIdx.x + tid] = d;
    }
    if (sm.pos[0] >= sm.pos[1]) return;  // the same for every thread

    if (tid == 0) {
        for (int s = 0; s < C::kKStages; ++s) {
            mbar_init(&sm.k_full[s], 1);
            mbar_init(&sm.k_empty[s], 1);
        }
        for (int s = 0; s < C::kVStages; ++s) {
            mbar_init(&sm.v_full[s], 1);
            mbar_init(&sm.v_empty[s], C::kHalf ? C::kConv / 32 : 1);
        }
        for (int s = 0; s < kMetas; ++s) {
            mbar_init(&sm.meta_full[s], 1);
            mbar_init(&sm.meta_empty[s], C::kSoft / 32);
        }
        for (int s = 0; s < kSegs; ++s) {
            mbar_init(&sm.seg_full[s], 1);
            mbar_init(&sm.seg_empty[s], (C::kSoft + C::kConv) / 32 + 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm.s_full[b], 1);
            mbar_init(&sm.p_ready[b], C::kSoft);
            mbar_init(&sm.pv_done[b], 1);
            if (C::kHalf) mbar_init(&sm.val_full[b], C::kConv);
        }
        mbar_init(&sm.raw_full, 1);
        mbar_init(&sm.raw_empty, C::kSoft / 32);
        mbar_init(&sm.q_ready, C::kSoft);
        sm.abort_flag = 0;
        mbar_init_fence();
        tma_prefetch_desc(&k_map);
        tma_prefetch_desc(&v_map);
    }
    if (warp == kIssuer) {
        tmem_alloc(&sm.tmem, C::kTmem);
        tmem_relinquish();
    }
    fence_async_shared();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    const Waiter wait = {&sm.abort_flag, status};

    if (warp == kProducer) {
        // ------------------------------------------------------------------------- producer
        int n = sm.at[0][0], h = sm.at[0][1], rt = sm.at[0][2], t0 = sm.at[0][3];
        int64_t left = sm.pos[1] - sm.pos[0];
        const int pp = kTileKeys / bs;
        int g = 0, k = 0;            // tiles and segments so far
        bool ok = true;
        Run r = {0, 0, 0};
        int loaded = -1;
        while (left > 0 && ok) {
            if (loaded != n) {
                r = load_run(a, n, nullptr);
                loaded = n;
            }
            if (r.len == 0) {
                ++n;
                h = rt = t0 = 0;
                continue;
            }
            const int u = unit_tiles<R>(r, group, rt), keys = unit_keys<R>(r, group, rt);
            const int t1 = (int)min((int64_t)u, t0 + left);
            left -= t1 - t0;
            // hand the segment over
            const int sk = k % kSegs;
            if (k >= kSegs) ok = wait(&sm.seg_empty[sk], (k / kSegs - 1) & 1);
            if (!ok) break;
            const int row0 = rt * R, rows = min(R, r.len * group - row0);
            const int slot = t0 == 0 && t1 == u ? -1 : 2 * (int)blockIdx.x + (t0 == 0);
            if (lane == 0) {
                Seg s = {};
                s.n = n;
                s.q0 = r.q0;
                s.head = h;
                s.row0 = row0;
                s.rows = rows;
                s.tile0 = t0;
                s.tile1 = keys > 0 ? t1 : t0;
                s.keys = keys;
                s.lim0 = r.ctx - r.len + 1;
                s.slot = slot;
                sm.segs[sk] = s;
                mbar_arrive(&sm.seg_full[sk]);
                if (slot >= 0) {
                    PartDesc d = {};
                    d.valid = 1;
                    d.n = n;
                    d.head = h;
                    d.rt = rt;
                    d.ends = t1 == u;
                    descs[slot] = d;
                }
            }
            // its rows of q, token by token
            if (k >= 1) ok = wait(&sm.raw_empty, (k - 1) & 1);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&sm.raw_full, (uint32_t)rows * 256);
            __syncwarp();
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
            for (int tk = row0 / group + lane; tk * group < row0 + rows; tk += 32) {
                const int ra = max(row0, tk * group), rb = min(row0 + rows, (tk + 1) * group);
                bulk_load(smem + C::kOffRaw + (ra - row0) * 256,
                          q + (int64_t)(r.q0 + tk) * a.q_stride + (h * group + ra - tk * group) * kDim,
                          (uint32_t)(rb - ra) * 256, &sm.raw_full);
            }
            ++k;
            // its tiles.  Lane l < pp has page l of a tile; tables are read two tiles ahead and
            // scales one, while the waits below pass.
            if (keys > 0) {
                const int32_t* table = a.tables + (int64_t)n * a.width;
                const int pages = (keys + bs - 1) / bs;
                auto page_of = [&](int t) {
                    const int b = t * pp + lane;
                    return lane < pp && t < t1 && b < pages ? table[b] : -2;
                };
                auto checked = [&](int id) {
                    if (id != -2 && (id < 0 || id >= a.num_pages)) {
                        report_status(status, KDA_ERR_INVALID_ARG);
                        return a.num_pages;  // outside the tensor map: zeros
                    }
                    return id;
                };
                auto scales_of = [&](int id) {
                    float2 s = make_float2(0.f, 1.f);
                    if (id >= 0 && id < a.num_pages) {
                        const int64_t ph = (int64_t)id * a.kv_heads + h;
                        s = make_float2(a.k_scale[ph], a.v_scale[ph]);
                    }
                    return s;
                };
                int id = checked(page_of(t0));
                int next = page_of(t0 + 1);
                float2 sc = scales_of(id);
                for (int t = t0; t < t1 && ok; ++t, ++g) {
                    const int sk = g % C::kKStages, sv = g % C::kVStages, me = g % kMetas;
                    const int live = min(pp, pages - t * pp);  // pages of this tile with keys
                    next = checked(next);
                    const float2 sc_next = scales_of(next);
                    const int after = page_of(t + 2);
                    if (g >= C::kKStages) ok = wait(&sm.k_empty[sk], (uint32_t)(g / C::kKStages - 1) & 1);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&sm.k_full[sk], (uint32_t)(live * bs * kDim));
                    __syncwarp();
                    if (lane < live)
                        tma_load_3d(smem + C::kOffK + sk * kTileBytes + lane * bs * kDim, &k_map,
                                    &sm.k_full[sk], 0, h * bs, id);
                    if (g >= kMetas) ok = wait(&sm.meta_empty[me], (uint32_t)(g / kMetas - 1) & 1);
                    if (!ok) break;
                    if (lane < kMaxTilePages) sm.meta[me][lane] = sc;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.meta_full[me]);
                    if (g >= C::kVStages) ok = wait(&sm.v_empty[sv], (uint32_t)(g / C::kVStages - 1) & 1);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&sm.v_full[sv], (uint32_t)(live * bs * kDim));
                    __syncwarp();
                    if (lane < live)
                        tma_load_3d(smem + C::kOffV + sv * kTileBytes + lane * bs * kDim, &v_map,
                                    &sm.v_full[sv], 0, h * bs, id);
                    id = next;
                    next = after;
                    sc = sc_next;
                }
            }
            t0 = 0;
            if (++rt == row_tiles<R>(r, group)) {
                rt = 0;
                if (++h == a.kv_heads) {
                    h = 0;
                    ++n;
                }
            }
        }
        if (ok) {
            const int sk = k % kSegs;
            if (k >= kSegs) ok = wait(&sm.seg_empty[sk], (k / kSegs - 1) & 1);
            if (ok && lane == 0) {
                sm.segs[sk].n = -1;
                mbar_arrive(&sm.seg_full[sk]);
            }
        }
        // every copy has landed before the CTA may end: the consumers waited for them all, unless
        // a wait gave up
        if (*static_cast<volatile int32_t*>(&sm.abort_flag)) {
            for (int i = max(0, g - C::kKStages); i <= g; ++i)
                mbar_wait(&sm.k_full[i % C::kKStages], (uint32_t)(i / C::kKStages) & 1, kAttnWaitLimit / 8);
            for (int i = max(0, g - C::kVStages); i <= g; ++i)
                mbar_wait(&sm.v_full[i % C::kVStages], (uint32_t)(i / C::kVStages) & 1, kAttnWaitLimit / 8);
            if (k > 0) mbar_wait(&sm.raw_full, (k - 1) & 1, kAttnWaitLimit / 8);
        }
    } else if (warp == kIssuer) {
        // ------------------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            constexpr uint32_t kIdQ = idesc_zero(C::kNQ, false, false);
            constexpr uint32_t kIdP = idesc_zero(C::kNP, true, true);  // f16's code is e4m3's: 0
            const uint32_t base = saddr(smem), o_col = tmem + 2 * C::kNQ;
            const uint64_t q_desc = smem_desc(base + C::kOffQ, 16, 1024);
            auto scores = [&](int g) {
                const int s = g % C::kKStages;
                if (!wait(&sm.k_full[s], (uint32_t)(g / C::kKStages) & 1)) return false;
                tc_fence_after();
                const uint64_t k_desc = smem_desc(base + C::kOffK + s * kTileBytes, 16, 1024);
#pragma unroll
                for (int i = 0; i < 4; ++i)  // 32 channels (32 bytes of a swizzled row) each
                    mma_f8(tmem + (g & 1) * C::kNQ, k_desc + 2 * i, q_desc + 2 * i, kIdQ, i > 0);
                mma_commit(&sm.k_empty[s]);
                mma_commit(&sm.s_full[g & 1]);
                return true;
            };
            auto sums = [&](int g, bool first) {
                const int b = g & 1, s = g % C::kVStages;
                if constexpr (C::kHalf) {
                    if (!wait(&sm.val_full[b], (uint32_t)(g >> 1) & 1)) return false;
                } else {
                    if (!wait(&sm.v_full[s], (uint32_t)(g / C::kVStages) & 1)) return false;
                }
                if (!wait(&sm.p_ready[b], (uint32_t)(g >> 1) & 1)) return false;
                tc_fence_after();
                const uint64_t p_desc = smem_desc(base + C::kOffP + b * C::kPBytes, 16384, 1024);
                if constexpr (C::kHalf) {
                    const uint64_t v_desc = smem_desc(base + C::kOffVal + b * C::kValBytes, 16384, 1024);
#pragma unroll
                    for (int i = 0; i < 8; ++i)  // 16 keys (16 rows of 128 bytes) each
                        mma_ss(o_col, v_desc + 128 * i, p_desc + 128 * i, kIdP, !first || i > 0);
                } else {
                    const uint64_t v_desc = smem_desc(base + C::kOffV + s * kTileBytes, 16384, 1024);
#pragma unroll
                    for (int i = 0; i < 4; ++i)  // 32 keys (32 rows of 128 bytes) each
                        mma_f8(o_col, v_desc + 256 * i, p_desc + 256 * i, kIdP, !first || i > 0);
                    mma_commit(&sm.v_empty[s]);
                }
                mma_commit(&sm.pv_done[b]);
                return true;
            };
            int g = 0, before = 0;  // tiles so far; tiles of the last segment, whose last is open
            for (int k = 0;; ++k) {
                if (!wait(&sm.seg_full[k % kSegs], (uint32_t)(k / kSegs) & 1)) break;
                const int n = sm.segs[k % kSegs].n;
                const int tiles = sm.segs[k % kSegs].tile1 - sm.segs[k % kSegs].tile0;
                if (before > 0 && !sums(g - 1, before == 1)) break;
                before = 0;
                if (n < 0) break;
                mbar_arrive(&sm.seg_empty[k % kSegs]);
                if (!wait(&sm.q_ready, k & 1)) break;
                tc_fence_after();
                bool ok = true;
                for (int i = 0; i < tiles && ok; ++i, ++g) {
                    ok = scores(g);
                    if (ok && i > 0) ok = sums(g - 1, i == 1);
                }
                if (!ok) break;
                before = tiles;
            }
        }
        __syncwarp();
    } else if (C::kHalf && warp >= C::kSoft / 32) {
        // ------------------------------------------------- values to f16, one key's row a thread
        const int key = tid - C::kSoft;
        bool ok = true;
        int g = 0;
        for (int k = 0;; ++k) {
            ok &= wait(&sm.seg_full[k % kSegs], (uint32_t)(k / kSegs) & 1);
            int32_t* first_nan = sm.first_nan[k % kSegs];
            first_nan[key] = INT32_MAX;
            if (conv_any(!ok)) break;  // a wait gave up: the four warps leave together
            const Seg& seg = sm.segs[k % kSegs];
            if (seg.n < 0) break;
            const int lim_min = seg.lim0 + seg.row0 / group, keys = seg.keys, tile1 = seg.tile1;
            int t = seg.tile0;
            for (; t < tile1; ++t, ++g) {
                const int b = g & 1, s = g % C::kVStages;
                if (!(ok = wait(&sm.v_full[s], (uint32_t)(g / C::kVStages) & 1))) break;
                if (g >= 2 && !(ok = wait(&sm.pv_done[b], (uint32_t)((g >> 1) - 1) & 1))) break;
                const unsigned char* row = smem + C::kOffV + s * kTileBytes + key * kDim;
                unsigned char* to = smem + C::kOffVal + b * C::kValBytes + key * 128;
                const int pos = t * kTileKeys + key;
                const bool cut = (t + 1) * kTileKeys > lim_min;
                uint4 v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = *reinterpret_cast<const uint4*>(row + ((j ^ (key & 7)) << 4));
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.v_empty[s]);
                if (cut) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) mask_values(v[j], pos < keys, pos, first_nan + j * 16);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v[j]);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t w0 = w[2 * half], w1 = w[2 * half + 1];
                        const int c = 2 * j + half;  // 8 channels: 16 bytes
                        *reinterpret_cast<uint4*>(to + (c >> 3) * 16384 + (((c & 7) ^ (key & 7)) << 4)) =
                            make_uint4(e4m3_to_half2((uint16_t)w0), e4m3_to_half2((uint16_t)(w0 >> 16)),
                                       e4m3_to_half2((uint16_t)w1), e4m3_to_half2((uint16_t)(w1 >> 16)));
                    }
                }
                fence_async_shared();
                mbar_arrive(&sm.val_full[b]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.seg_empty[k % kSegs]);
        }
    } else {
        // --------------------------------------------------------- scores, weights and outputs
        // Warpgroup wg has rows r0 .. r0 + kRW - 1 of the tile; its thread `key` has one key of the
        // tile (a TMEM lane) for the weights and one channel for the outputs.
        constexpr int kRW = C::kRW;
        const int wg = warp >> 2, key = tid & 127, r0 = wg * kRW;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // TMEM lane 32 * (warp % 4)
        const uint32_t o_col = lanes + 2 * C::kNQ + r0;
        const int page_at = key / bs;
        bool dead = false;  // a wait gave up: run on to where all warpgroups can leave together
        float qc = 0.f;     // score scale of the segment: sm_scale log2 e / s

        // Rows of q of segment k as two e4m3 terms, scaled by one power of two s so that the
        // largest lies in [128, 256).  Returns 1 / s.  An item is 16 channels of a row.
        constexpr int kItems = (R * 8 + C::kSoft - 1) / C::kSoft;
        auto convert = [&](int k, const Seg& sg) {
            dead |= !wait(&sm.raw_full, k & 1);
            uint32_t mx = 0;
            uint4 x[kItems][2];
#pragma unroll
            for (int it = 0; it < kItems; ++it) {
                const int row = (it * C::kSoft + tid) >> 3, j = tid & 7;
                x[it][0] = x[it][1] = make_uint4(0, 0, 0, 0);
                if (row < sg.rows) {
                    const uint4* p = reinterpret_cast<const uint4*>(smem + C::kOffRaw + row * 256 + j * 32);
                    x[it][0] = p[0];
                    x[it][1] = p[1];
                }
                const uint32_t* w = reinterpret_cast<const uint32_t*>(x[it]);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint32_t lo = w[c] & 0x7fffu, hi = (w[c] >> 16) & 0x7fffu;
                    mx = max(mx, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
                }
            }
            mx = __reduce_max_sync(~0u, mx);
            if (lane == 0) sm.qred[warp] = mx;
            if (tid < R) {
                const int at = sg.row0 + tid, tok = at / group;
                sm.lim[k & 1][tid] = tid < sg.rows ? sg.lim0 + tok : 0;
                sm.orow[k & 1][tid] = (sg.q0 + tok) * a.heads + sg.head * group + at % group;
            }
            all_any<C::kSoft>(false);
#pragma unroll
            for (int i = 0; i < C::kSoft / 32; ++i) mx = max(mx, sm.qred[i]);
            // exponents outside +-100 are left alone: such rows have scores of 0 or infinity
            const int e = mx == 0 ? 127 : min(max((int)(mx >> 7), 27), 227);
            const float s = __int_as_float((127 + 134 - e) << 23);
#pragma unroll
            for (int it = 0; it < kItems; ++it) {
                const int row = (it * C::kSoft + tid) >> 3, j = tid & 7;
                const uint32_t* w = reinterpret_cast<const uint32_t*>(x[it]);
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    float y0 = __uint_as_float(w[c] << 16) * s, y1 = __uint_as_float(w[c] & 0xffff0000u) * s;
                    if (isinf(y0)) y0 = NAN;
                    if (isinf(y1)) y1 = NAN;
                    const uint16_t h2 = float2_to_e4m3(y0, y1);
                    const float2 b = __half22float2(as_half2(e4m3_to_half2(h2)));
                    const uint16_t l2 = float2_to_e4m3((y0 - b.x) * 16.f, (y1 - b.y) * 16.f);
                    if (c & 1) {
                        hi[c >> 1] |= (uint32_t)h2 << 16;
                        lo[c >> 1] |= (uint32_t)l2 << 16;
                    } else {
                        hi[c >> 1] = h2;
                        lo[c >> 1] = l2;
                    }
                }
                if (row < R) {
                    unsigned char* q = smem + C::kOffQ;
                    const int rl = R + row;
                    *reinterpret_cast<uint4*>(q + row * 128 + ((j ^ (row & 7)) << 4)) =
                        make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(q + rl * 128 + ((j ^ (rl & 7)) << 4)) =
                        make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            fence_async_shared();
            mbar_arrive(&sm.q_ready);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.raw_empty);
            return __int_as_float((127 - 134 + e) << 23);
        };

        dead |= !wait(&sm.seg_full[0], 0);
        if (!all_any<C::kSoft>(dead)) {
            qc = convert(0, sm.segs[0]) * a.sm_scale * kLog2e;
            int g = 0;
            for (int k = 0;; ++k) {
                if (key < kRW) sm.mref[r0 + key] = 0.f;
                if (!C::kHalf && tid < kDim) sm.first_nan[k % kSegs][tid] = INT32_MAX;
                float l[kRW];
#pragma unroll
                for (int r = 0; r < kRW; ++r) l[r] = 0.f;
                all_any<C::kSoft>(false);
                // the segment's fields stay in shared memory until it is given back
                const Seg& seg = sm.segs[k % kSegs];
                const int lim_min = seg.lim0 + seg.row0 / group, keys = seg.keys, tile1 = seg.tile1;
                const int32_t* lim = sm.lim[k & 1] + r0;
                bool first = true;
                for (int t = seg.tile0; t < tile1; ++t, ++g, first = false) {
                    const int b = g & 1, me = g % kMetas;
                    dead |= !wait(&sm.meta_full[me], (uint32_t)(g / kMetas) & 1);
                    const float2 sc = sm.meta[me][page_at];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.meta_empty[me]);
                    const int pos = t * kTileKeys + key;
                    const bool in = pos < keys;
                    const float c1 = in ? sc.x * qc : 0.f, c2 = c1 * 0.0625f;
                    const float lvs = in ? lg2(sc.y) : 0.f, inv = in ? rcp(sc.y) : 0.f;
                    const bool cut = (t + 1) * kTileKeys > lim_min;  // some row does not see all
                    dead |= !wait(&sm.s_full[b], (uint32_t)(g >> 1) & 1);
                    tc_fence_after();
                    // scores in base 2 with the value scale, less their row's reference
                    float x[kRW];
                    {
                        const float2 cc1 = make_float2(c1, c1), cc2 = make_float2(c2, c2);
                        const float2 lv = make_float2(lvs, lvs);
                        constexpr int kN = kRW < 16 ? kRW : 16;
#pragma unroll
                        for (int q = 0; q < kRW; q += kN) {
                            float u[2][kN];
                            tmem_ld_start<kN>(lanes + b * C::kNQ + r0 + q, u[0]);
                            tmem_ld_start<kN>(lanes + b * C::kNQ + R + r0 + q, u[1]);
                            tmem_ld_wait<kN, 2>(u);
#pragma unroll
                            for (int i = 0; i < kN; i += 2) {
                                const float2 m = *reinterpret_cast<const float2*>(sm.mref + r0 + q + i);
                                const float2 y = fma_f32x2(
                                    make_float2(u[0][i], u[0][i + 1]), cc1,
                                    fma_f32x2(make_float2(u[1][i], u[1][i + 1]), cc2, add_f32x2(lv, m)));
                                x[q + i] = y.x;
                                x[q + i + 1] = y.y;
                            }
                        }
                    }
                    if (cut) {
#pragma unroll
                        for (int r = 0; r < kRW; r += 4) {
                            const int4 m = *reinterpret_cast<const int4*>(lim + r);
                            x[r] = pos < m.x ? x[r] : -INFINITY;
                            x[r + 1] = pos < m.y ? x[r + 1] : -INFINITY;
                            x[r + 2] = pos < m.z ? x[r + 2] : -INFINITY;
                            x[r + 3] = pos < m.w ? x[r + 3] : -INFINITY;
                        }
                        if (!C::kHalf && wg == 0) {
                            const int s = g % C::kVStages;
                            dead |= !wait(&sm.v_full[s], (uint32_t)(g / C::kVStages) & 1);
                            unsigned char* row = smem + C::kOffV + s * kTileBytes + key * kDim;
#pragma unroll 1
                            for (int j = 0; j < 8; ++j) {
                                uint4* p = reinterpret_cast<uint4*>(row + ((j ^ (key & 7)) << 4));
                                uint4 v = *p;
                                if (mask_values(v, in, pos, sm.first_nan[k % kSegs] + j * 16)) *p = v;
                            }
                        }
                    }
                    // does any score exceed its row's reference by too much?
                    float over = x[0];
#pragma unroll
                    for (int r = 1; r < kRW; ++r) over = fmaxf(over, x[r]);
                    if (group_any(wg, over > C::kPeak + C::kSlack || first)) {
#pragma unroll
                        for (int r = 0; r < kRW; ++r) {
                            const int m = __reduce_max_sync(~0u, ordered(x[r]));
                            if (lane == r) sm.red[warp & 3][r0 + r] = unordered(m);
                        }
                        group_sync(wg);
                        if (key < kRW) {
                            // the reference rises by what the largest score is above 2^kPeak; the
                            // segment's first tile sets it.  A row that sees no key there sees none
                            // in the segment.
                            const int r = r0 + key;
                            const float top = fmaxf(fmaxf(sm.red[0][r], sm.red[1][r]),
                                                    fmaxf(sm.red[2][r], sm.red[3][r]));
                            float up = first ? top - C::kPeak : fmaxf(top - C::kPeak, 0.f);
                            if (!(up > -1e37f)) up = first ? kNoRef : 0.f;
                            sm.fac[r] = up;
                            sm.mref[r] -= up;
                        }
                        if (!first) {
                            dead |= !wait(&sm.pv_done[(g - 1) & 1], (uint32_t)((g - 1) >> 1) & 1);
                            tc_fence_after();
                        }
                        group_sync(wg);
#pragma unroll
                        for (int r = 0; r < kRW; ++r) x[r] -= sm.fac[r0 + r];
                        if (!first) {
#pragma unroll
                            for (int r = 0; r < kRW; ++r) l[r] *= ex2_approx(-sm.fac[r0 + r]);
#pragma unroll 1
                            for (int c = 0; c < C::kTerms * kRW; c += 8) {
                                const int col = c / kRW * R + c % kRW;
                                float o[1][8];
                                tmem_ld_start<8>(o_col + col, o[0]);
                                tmem_ld_wait<8, 1>(o);
#pragma unroll
                                for (int r = 0; r < 8; ++r) o[0][r] *= ex2_approx(-sm.fac[r0 + c % kRW + r]);
                                tmem_st8(o_col + col, o[0]);
                            }
                            tmem_st_wait();
                        }
                    }
                    // weights and their sums; into this key's row of P as f16 or three e4m3 terms
                    if (g >= 2) dead |= !wait(&sm.pv_done[b], (uint32_t)((g >> 1) - 1) & 1);
                    unsigned char* pt = smem + C::kOffP + b * C::kPBytes + key * 128;
                    auto p_chunk = [&](int byte) {  // 16 bytes of the row
                        return reinterpret_cast<uint4*>(pt + (((byte >> 4) ^ (key & 7)) << 4));
                    };
                    const float2 inv2 = make_float2(inv, inv);
                    uint32_t term[3][4];
#pragma unroll
                    for (int i = 0; i < kRW; i += 2) {
                        const float p0 = ex2_approx(x[i]), p1 = ex2_approx(x[i + 1]);
                        const float2 sum = fma_f32x2(make_float2(p0, p1), inv2, make_float2(l[i], l[i + 1]));
                        l[i] = sum.x;
                        l[i + 1] = sum.y;
                        const __half2 p = __floats2half2_rn(p0, p1);
                        if constexpr (C::kHalf) {
                            term[0][(i >> 1) & 3] = as_u32(p);
                            if ((i & 7) == 6)
                                *p_chunk((r0 + i - 6) * 2) = make_uint4(term[0][0], term[0][1], term[0][2], term[0][3]);
                        } else {
                            const uint16_t e0 = half2_to_e4m3(as_u32(p));
                            const __half2 d1 = __hsub2(p, as_half2(e4m3_to_half2(e0)));
                            const uint16_t e1 = half2_to_e4m3(as_u32(d1));
                            const __half2 d2 = __hsub2(d1, as_half2(e4m3_to_half2(e1)));
                            const uint16_t e2 = half2_to_e4m3(as_u32(__hmul2(d2, __float2half2_rn(512.f))));
                            const int w = i >> 2;
                            if (i & 2) {
                                term[0][w] |= (uint32_t)e0 << 16;
                                term[1][w] |= (uint32_t)e1 << 16;
                                term[2][w] |= (uint32_t)e2 << 16;
                            } else {
                                term[0][w] = e0;
                                term[1][w] = e1;
                                term[2][w] = e2;
                            }
                        }
                    }
                    if constexpr (R == 8) {
                        *p_chunk(0) = make_uint4(term[0][0], term[0][1], term[1][0], term[1][1]);
                        *p_chunk(16) = make_uint4(term[2][0], term[2][1], 0, 0);
                    } else if constexpr (!C::kHalf) {
#pragma unroll
                        for (int c = 0; c < 3; ++c)
                            *p_chunk(c * R + r0) = make_uint4(term[c][0], term[c][1], term[c][2], term[c][3]);
                    }
                    fence_async_shared();
                    tc_fence_before();
                    mbar_arrive(&sm.p_ready[b]);
                }
                // the next segment's q, so that its first scores run under this one's outputs
                const int kn = k + 1;
                dead |= !wait(&sm.seg_full[kn % kSegs], (uint32_t)(kn / kSegs) & 1);
                if (all_any<C::kSoft>(dead)) break;
                const bool more = sm.segs[kn % kSegs].n >= 0;
                if (more) qc = convert(kn, sm.segs[kn % kSegs]) * a.sm_scale * kLog2e;
                // outputs: thread = channel
                const bool some = !first;
                if (some) {
                    dead |= !wait(&sm.pv_done[(g - 1) & 1], (uint32_t)((g - 1) >> 1) & 1);
                    tc_fence_after();
                    const float mine = warp_sums<kRW>(l, lane);
                    if (lane < kRW) sm.red[warp & 3][r0 + lane] = mine;
                    group_sync(wg);
                    if (key < kRW) {
                        const int r = r0 + key;
                        const float sum = sm.red[0][r] + sm.red[1][r] + sm.red[2][r] + sm.red[3][r];
                        if (seg.slot >= 0) {
                            parts[seg.slot].m[r] = -sm.mref[r];
                            parts[seg.slot].l[r] = sum;
                            sm.fac[r] = 1.f;
                        } else {
                            sm.fac[r] = sum == 0.f ? 0.f : 1.f / sum;
                        }
                    }
                    group_sync(wg);
                }
                const int mine = seg.rows - r0;  // rows of this warpgroup that are there
                if (mine > 0) {
                    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
                    const int32_t* orow = sm.orow[k & 1] + r0;
                    const int nan_from = sm.first_nan[k % kSegs][key];
#pragma unroll 1
                    for (int q = 0; q < kRW; q += 8) {
                        if (q >= mine) break;
                        float o[C::kTerms][8];
                        if (some) {
#pragma unroll
                            for (int c = 0; c < C::kTerms; ++c) tmem_ld_start<8>(o_col + c * R + q, o[c]);
                            tmem_ld_wait<8, C::kTerms>(o);
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (q + i >= mine) break;
                            float y = 0.f;
                            if (some) {
                                y = o[0][i];
                                if constexpr (C::kTerms == 3) y += o[1][i] + o[2][i] * 0x1p-9f;
                                y *= sm.fac[r0 + q + i];
                            }
                            if (lim[q + i] > nan_from) y = NAN;
                            if (seg.slot >= 0) parts[seg.slot].o[r0 + q + i][key] = y;
                            else out[(int64_t)orow[q + i] * kDim + key] = __float2bfloat16_rn(y);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.seg_empty[k % kSegs]);
                if (!more) break;
                all_any<C::kSoft>(false);  // mref, fac, the sums and first_nan are free again
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kIssuer) tmem_dealloc(tmem, C::kTmem);
}

// Joins the partial results of the units that more than one CTA worked on, in key order.  Unit u's
// parts are the last of the CTA that began it and the first of those that went on.  Every block
// lists the units (the descriptors are few) and takes its share of the items: four rows, one a
// warp, of a unit in up to kJoinParts parts, else one row whose parts the four warps share.
constexpr int kJoinThreads = 128, kJoinWarps = kJoinThreads / 32, kJoinParts = 16;
template <int R>
__global__ void __launch_bounds__(kJoinThreads) paged_attention_join_kernel(const AttnArgs a, int ctas) {
    constexpr int kMaxCtas = 2 * kPlanSMs, kPer = (kMaxCtas + kJoinThreads - 1) / kJoinThreads;
    __shared__ uint32_t ends[kMaxCtas / 32 + 1];  // CTAs whose first part ends its unit
    __shared__ int32_t first_item[kMaxCtas + 1], sums[kJoinWarps];
    __shared__ float part_m[kJoinWarps], part_l[kJoinWarps];
    __shared__ float4 part_o[kJoinWarps][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PartDesc* descs = static_cast<const PartDesc*>(a.workspace);
    const Part<R>* parts = reinterpret_cast<const Part<R>*>(static_cast<const char*>(a.workspace) +
                                                            (size_t)ctas * 2 * sizeof(PartDesc));
    bool begins[kPer];
    bool any = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int c = i * kJoinThreads + tid;
        bool end = c >= ctas - 1;
        begins[i] = false;
        if (c < ctas) {
            const int2 d = *reinterpret_cast<const int2*>(&descs[2 * c].valid);
            end |= d.x && descs[2 * c].ends;
            begins[i] = descs[2 * c + 1].valid;
            any |= begins[i];
        }
        const uint32_t m = __ballot_sync(~0u, end);
        if (lane == 0 && i * kJoinThreads + warp * 32 <= kMaxCtas) ends[i * kJoinWarps + warp] = m;
    }
    if (!__syncthreads_or(any)) return;
    // items before each unit: a scan over the CTAs, 32 * kJoinWarps at a time
    int items = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int c = i * kJoinThreads + tid;
        int mine = 0;
        if (begins[i]) {
            int w = (c + 1) >> 5;
            uint32_t bits = ends[w] & (~0u << ((c + 1) & 31));
            while (bits == 0) bits = ends[++w];
            const int count = w * 32 + __ffs(bits) - c;
            mine = count <= kJoinParts ? R / 4 : R;
        }
        int in = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(~0u, in, d);
            if (lane >= d) in += y;
        }
        __syncthreads();
        if (lane == 31) sums[warp] = in;
        __syncthreads();
        int base = items;
        for (int w = 0; w < kJoinWarps; ++w) {
            if (w < warp) base += sums[w];
            items += sums[w];
        }
        if (c < ctas) first_item[c] = base + in - mine;
    }
    if (tid == 0) first_item[ctas] = items;
    __syncthreads();
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int c = seq_of_row(first_item, ctas, item);
        const PartDesc d = descs[2 * c + 1];
        int w = (c + 1) >> 5;
        uint32_t bits = ends[w] & (~0u << ((c + 1) & 31));
        while (bits == 0) bits = ends[++w];
        const int last = w * 32 + __ffs(bits) - 1, count = last - c + 1, at = item - first_item[c];
        const bool shared = count > kJoinParts;
        const int row = shared ? at : at * 4 + warp;
        const Run r = load_run(a, d.n, nullptr);
        const int group = a.heads / a.kv_heads, run_row = d.rt * R + row;
        const bool live = run_row < r.len * group;
        auto part = [&](int i) -> const Part<R>& { return parts[i == 0 ? 2 * c + 1 : 2 * (c + i)]; };
        float m = kNoRef, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (live) {
            // this warp's parts: all, or every kJoinWarps-th
            const int step = shared ? kJoinWarps : 1, from = shared ? warp : 0;
            const int mine = (count - from + step - 1) / step;
            for (int i = lane; i < mine; i += 32) m = fmaxf(m, part(from + i * step).m[row]);
#pragma unroll
            for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, x));
            for (int i0 = 0; i0 < mine; i0 += 32) {
                const int i = min(i0 + lane, mine - 1), n = min(mine - i0, 32);
                const Part<R>& p = part(from + i * step);
                const float f = ex2_approx(p.m[row] - m), fl = lane < n ? f * p.l[row] : 0.f;
#pragma unroll 8
                for (int j = 0; j < n; ++j) {
                    const float x = __shfl_sync(~0u, f, j);
                    const float4 y = *reinterpret_cast<const float4*>(
                        &part(from + (i0 + j) * step).o[row][lane * 4]);
                    l += __shfl_sync(~0u, fl, j);
                    o.x += x * y.x;
                    o.y += x * y.y;
                    o.z += x * y.z;
                    o.w += x * y.w;
                }
            }
        }
        if (shared) {
            part_o[warp][lane] = o;
            if (lane == 0) {
                part_m[warp] = m;
                part_l[warp] = l;
            }
            __syncthreads();
            if (warp == 0) {
                m = fmaxf(fmaxf(part_m[0], part_m[1]), fmaxf(part_m[2], part_m[3]));
                l = 0.f;
                o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int j = 0; j < kJoinWarps; ++j) {
                    const float x = ex2_approx(part_m[j] - m);
                    l += x * part_l[j];
                    o.x += x * part_o[j][lane].x;
                    o.y += x * part_o[j][lane].y;
                    o.z += x * part_o[j][lane].z;
                    o.w += x * part_o[j][lane].w;
                }
            }
            __syncthreads();
        }
        if (live && (!shared || warp == 0)) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const int64_t to = (int64_t)(r.q0 + run_row / group) * a.heads + d.head * group + run_row % group;
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + to * kDim + lane * 4) =
                make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        }
    }
}

// ---------------------------------------------------------------------------------------- host
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// 3-D map over [num_pages][kv_heads * page_size][128] bytes, box = one head's page.
bool make_map(CUtensorMap* map, const void* base, const AttnArgs& a) {
    auto enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t rows = (cuuint64_t)a.kv_heads * a.page_size;
    cuuint64_t dims[3] = {(cuuint64_t)kDim, rows, (cuuint64_t)a.num_pages};
    cuuint64_t strides[2] = {(cuuint64_t)kDim, rows * kDim};
    cuuint32_t box[3] = {(cuuint32_t)kDim, (cuuint32_t)a.page_size, 1};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of a tile: the least that holds a key head's rows of the longest run, at most 64.
int tile_rows(int heads, int kv_heads, int max_run) {
    const int64_t rows = (int64_t)(heads / kv_heads) * std::max(max_run, 1);
    return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}
template <int R>
constexpr int ctas_of() { return kPlanSMs * Cfg<R>::kCtasPerSm; }
template <int R>
constexpr size_t workspace_of() { return (size_t)ctas_of<R>() * 2 * (sizeof(PartDesc) + sizeof(Part<R>)); }

template <int R>
cudaError_t launch_rows(const AttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, int* status,
                        cudaStream_t stream) {
    // the shared memory of a kernel is raised once per device
    static std::atomic<uint64_t> raised{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(raised.load() & bit)) {
        e = cudaFuncSetAttribute(paged_attention_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem_bytes<R>());
        if (e != cudaSuccess) return e;
        raised.fetch_or(bit);
    }
    paged_attention_kernel<R><<<ctas_of<R>(), Cfg<R>::kThreads, smem_bytes<R>(), stream>>>(a, km, vm, status);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * kPlanSMs);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_attention_join_kernel<R>, a, ctas_of<R>());
}

}  // namespace

size_t paged_attention_workspace(int32_t heads, int32_t kv_heads, int32_t max_run) {
    switch (tile_rows(heads, kv_heads, max_run)) {
        case 8: return workspace_of<8>();
        case 16: return workspace_of<16>();
        case 32: return workspace_of<32>();
        default: return workspace_of<64>();
    }
}

cudaError_t launch_paged_attention(const AttnArgs& a, int* status, cudaStream_t stream,
                                   uint64_t* launches) {
    CUtensorMap km, vm;
    if (!make_map(&km, a.k_cache, a) || !make_map(&vm, a.v_cache, a)) return cudaErrorInvalidValue;
    *launches += 2;
    switch (tile_rows(a.heads, a.kv_heads, a.max_run)) {
        case 8: return launch_rows<8>(a, km, vm, status, stream);
        case 16: return launch_rows<16>(a, km, vm, status, stream);
        case 32: return launch_rows<32>(a, km, vm, status, stream);
        default: return launch_rows<64>(a, km, vm, status, stream);
    }
}

}  // namespace kda
