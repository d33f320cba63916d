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
//   O^T [128 channels x 3R] += V^T [128 x 128] [P_0 P_1 P_2]    p = P_0 + P_1 / 2^4 + P_2 / 2^9: 11
//                        bits for weights within 2^13 of the largest, 2^-25 of it at the least
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
// Roles of a CTA's six warps:
//   0-3  scores -> weights, one thread per key of the tile (its TMEM lane), and the outputs, one
//        thread per channel.  Row maxima are not taken per tile: weights are formed against a
//        reference that a row's scores may exceed by up to 2^2.5 before the four warps agree (one
//        barrier with a vote) to raise it and rescale O^T, which after the first tile is rare.
//   4    producer: work list, page tables and scales a tile ahead, TMA of K, V and raw q
//   5    issues the MMAs: scores of tile j + 1 before the weighted sum of tile j
//
// Masked places.  Keys beyond a row's limit get weight 0.  Values beyond the request's context are
// zeroed in shared memory (0 * NaN), and a NaN value inside it is replaced by 0 in tiles where some
// row may not see it and put back into the rows that do.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "kda_common.cuh"
#include "kda_paged.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int kTileKeys = 128;
constexpr int kTileBytes = kTileKeys * kDim;  // one K or V tile, e4m3
constexpr int kAttnThreads = 192;
constexpr int kSegs = 4;                      // work descriptors in flight
constexpr int kMaxTilePages = 8;              // pages of 16 tokens in a tile
constexpr int kSnapUnit = 4, kSnapEdge = 2;   // units this short, and cuts this near, are not cut
constexpr int kGrainTiles = 4;                // least share of a CTA
constexpr long long kAttnWaitLimit = 4000000000LL;  // clock cycles (about 2 s)
// Weights are 2^6 at the reference and at most 2^8.5 = 362 < 448 above it.
constexpr float kPeak = 6.f, kSlack = 2.5f;
constexpr float kNoRef = -1e37f;              // reference of a row that has seen no key
constexpr float kLog2e = 1.4426950408889634f;

template <int R>
struct Cfg {
    static constexpr int kNQ = 2 * R;                       // columns of a score tile
    static constexpr int kNP = (3 * R + 15) / 16 * 16;      // columns of the output tile
    static constexpr int kCtasPerSm = R <= 16 ? 2 : 1;
    static constexpr int kStages = R <= 16 ? 2 : R == 32 ? 5 : 3;
    static constexpr int kTmem = R == 8 ? 64 : R == 16 ? 128 : R == 32 ? 256 : 512;
    static constexpr int kPBytes = kNP > 128 ? 2 * 16384 : 16384;
    static constexpr uint32_t kOffK = 0;
    static constexpr uint32_t kOffV = kOffK + kStages * kTileBytes;
    static constexpr uint32_t kOffP = kOffV + kStages * kTileBytes;
    static constexpr uint32_t kOffQ = kOffP + 2 * kPBytes;
    static constexpr uint32_t kOffRaw = kOffQ + kNQ * 128;
    static constexpr uint32_t kOffSmall = kOffRaw + R * 256;
    static_assert(2 * kNQ + kNP <= kTmem, "tensor memory columns");
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
    int32_t first_nan[kDim];
    float2 meta[Cfg<R>::kStages][kMaxTilePages];
    Seg segs[kSegs];
    uint64_t k_full[Cfg<R>::kStages], k_empty[Cfg<R>::kStages];
    uint64_t v_full[Cfg<R>::kStages], v_empty[Cfg<R>::kStages], meta_full[Cfg<R>::kStages];
    uint64_t seg_full[kSegs], seg_empty[kSegs];
    uint64_t s_full[2], p_ready[2], pv_done[2], raw_full, raw_empty, q_ready;
    uint32_t qred[4];
    uint32_t tmem;
    int32_t abort_flag;
    // the share: first unit and tile, and how many tiles
    int64_t scan[kAttnThreads / 32];
    int64_t total;
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

__device__ __forceinline__ void group_sync() {  // warps 0-3
    asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
}
__device__ __forceinline__ bool group_any(bool x) {  // warps 0-3: does any thread say so
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
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
// e4m3 x e4m3 -> fp32, M = 128.
__host__ __device__ constexpr uint32_t idesc_e4m3(int N, bool a_mn_major, bool b_mn_major) {
    return (1u << 4) | ((uint32_t)a_mn_major << 15) | ((uint32_t)b_mn_major << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
template <int C>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[C]) {
    if constexpr (C == 16) tmem_ld16(addr, r);
    else if constexpr (C == 32) tmem_ld32(addr, r);
    else tmem_ld64(addr, r);
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
// Order-preserving map of floats to integers (for an integer maximum over a warp).
__device__ __forceinline__ int32_t ordered(float x) {
    const int32_t i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int32_t i) {
    return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}

// Sums over the warp of R values per lane; lane l < R (R < 32: l % R) gets the sum of value l, for
// R = 64 the sums of values l and 32 + l.
template <int R>
__device__ __forceinline__ void warp_sums(float (&v)[R], int lane) {
    constexpr int kN = R < 32 ? R : 32;
#pragma unroll
    for (int b = 0; b < R; b += 32) {
#pragma unroll
        for (int off = kN / 2; off >= 1; off >>= 1) {
            const bool up = lane & off;
#pragma unroll
            for (int i = 0; i < off; ++i) {
                const float keep = up ? v[b + i + off] : v[b + i];
                const float send = up ? v[b + i] : v[b + i + off];
                v[b + i] = keep + __shfl_xor_sync(~0u, send, off);
            }
        }
#pragma unroll
        for (int off = kN; off < 32; off <<= 1) v[b] += __shfl_xor_sync(~0u, v[b], off);
    }
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
    const int per = (N + kAttnThreads - 1) / kAttnThreads, n0 = min(tid * per, N), n1 = min(n0 + per, N);
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
    for (int w = 0; w < kAttnThreads / 32; ++w) {
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
__global__ void __launch_bounds__(kAttnThreads, Cfg<R>::kCtasPerSm)
paged_attention_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap k_map,
                       const __grid_constant__ CUtensorMap v_map, int* status) {
    using C = Cfg<R>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    Small<R>& sm = *reinterpret_cast<Small<R>*>(smem + C::kOffSmall);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&sm.k_full[s], 1);
            mbar_init(&sm.k_empty[s], 1);
            mbar_init(&sm.v_full[s], 1);
            mbar_init(&sm.v_empty[s], 1);
            mbar_init(&sm.meta_full[s], 1);
        }
        for (int s = 0; s < kSegs; ++s) {
            mbar_init(&sm.seg_full[s], 1);
            mbar_init(&sm.seg_empty[s], 5);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm.s_full[b], 1);
            mbar_init(&sm.p_ready[b], 128);
            mbar_init(&sm.pv_done[b], 1);
        }
        mbar_init(&sm.raw_full, 1);
        mbar_init(&sm.raw_empty, 4);
        mbar_init(&sm.q_ready, 128);
        sm.abort_flag = 0;
        mbar_init_fence();
        tma_prefetch_desc(&k_map);
        tma_prefetch_desc(&v_map);
    }
    if (warp == 5) {
        tmem_alloc(&sm.tmem, C::kTmem);
        tmem_relinquish();
    }
    fence_async_shared();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    const Waiter wait = {&sm.abort_flag, status};

    if (warp == 4) {
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
                    const int s = g % C::kStages;
                    const uint32_t ph = (uint32_t)(g / C::kStages) & 1;
                    const int live = min(pp, pages - t * pp);  // pages of this tile with keys
                    next = checked(next);
                    const float2 sc_next = scales_of(next);
                    const int after = page_of(t + 2);
                    if (g >= C::kStages) ok = wait(&sm.k_empty[s], ph ^ 1);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&sm.k_full[s], (uint32_t)(live * bs * kDim));
                    __syncwarp();
                    if (lane < live)
                        tma_load_3d(smem + C::kOffK + s * kTileBytes + lane * bs * kDim, &k_map,
                                    &sm.k_full[s], 0, h * bs, id);
                    if (g >= C::kStages) ok = wait(&sm.v_empty[s], ph ^ 1);
                    if (!ok) break;
                    if (lane < kMaxTilePages) sm.meta[s][lane] = sc;
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sm.meta_full[s]);
                        mbar_arrive_expect_tx(&sm.v_full[s], (uint32_t)(live * bs * kDim));
                    }
                    __syncwarp();
                    if (lane < live)
                        tma_load_3d(smem + C::kOffV + s * kTileBytes + lane * bs * kDim, &v_map,
                                    &sm.v_full[s], 0, h * bs, id);
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
            for (int i = max(0, g - C::kStages); i <= g; ++i) {
                const int s = i % C::kStages;
                mbar_wait(&sm.k_full[s], (uint32_t)(i / C::kStages) & 1, kAttnWaitLimit / 8);
                mbar_wait(&sm.v_full[s], (uint32_t)(i / C::kStages) & 1, kAttnWaitLimit / 8);
            }
            if (k > 0) mbar_wait(&sm.raw_full, (k - 1) & 1, kAttnWaitLimit / 8);
        }
    } else if (warp == 5) {
        // ------------------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            constexpr uint32_t kIdQ = idesc_e4m3(C::kNQ, false, false);
            constexpr uint32_t kIdP = idesc_e4m3(C::kNP, true, true);
            const uint32_t base = saddr(smem), o_col = tmem + 2 * C::kNQ;
            const uint64_t q_desc = smem_desc(base + C::kOffQ, 16, 1024);
            auto scores = [&](int g) {
                const int s = g % C::kStages;
                if (!wait(&sm.k_full[s], (uint32_t)(g / C::kStages) & 1)) return false;
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
                const int s = g % C::kStages;
                if (!wait(&sm.v_full[s], (uint32_t)(g / C::kStages) & 1)) return false;
                if (!wait(&sm.p_ready[g & 1], (uint32_t)(g >> 1) & 1)) return false;
                tc_fence_after();
                const uint64_t v_desc = smem_desc(base + C::kOffV + s * kTileBytes, 16384, 1024);
                const uint64_t p_desc = smem_desc(base + C::kOffP + (g & 1) * C::kPBytes, 16384, 1024);
#pragma unroll
                for (int i = 0; i < 4; ++i)  // 32 keys (32 rows of 128 bytes) each
                    mma_f8(o_col, v_desc + 256 * i, p_desc + 256 * i, kIdP, !first || i > 0);
                mma_commit(&sm.v_empty[s]);
                mma_commit(&sm.pv_done[g & 1]);
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
    } else {
        // --------------------------------------------------------- scores, weights and outputs
        const uint32_t lanes = tmem + ((uint32_t)warp << 21);  // TMEM lane 32 * warp
        const uint32_t o_col = lanes + 2 * C::kNQ;
        bool dead = false;
        Seg seg;
        float qc = 0.f;  // score scale of the segment: sm_scale log2 e / s

        // Rows of q of segment k as two e4m3 terms, scaled by one power of two s so that the
        // largest lies in [128, 256).  Returns 1 / s.
        auto convert = [&](int k, const Seg& sg) {
            dead |= !wait(&sm.raw_full, k & 1);
            const unsigned char* raw = smem + C::kOffRaw;
            constexpr int kItems = (R * 8 + 127) / 128;  // 16 channels of a row each
            uint4 x[kItems][2];
            uint32_t mx = 0;
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                const int item = i * 128 + tid, row = item >> 3;
                x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
                if (row < sg.rows) {
                    const uint4* p = reinterpret_cast<const uint4*>(raw + row * 256 + (item & 7) * 32);
                    x[i][0] = p[0];
                    x[i][1] = p[1];
                }
                const uint32_t* w = reinterpret_cast<const uint32_t*>(x[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t lo = w[j] & 0x7fffu, hi = (w[j] >> 16) & 0x7fffu;
                    mx = max(mx, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
                }
            }
            mx = __reduce_max_sync(~0u, mx);
            if (lane == 0) sm.qred[warp] = mx;
            if (tid < R) {
                const int row = sg.row0 + tid, tok = row / group;
                sm.lim[k & 1][tid] = tid < sg.rows ? sg.lim0 + tok : 0;
                sm.orow[k & 1][tid] = (sg.q0 + tok) * a.heads + sg.head * group + row % group;
            }
            group_sync();
            mx = max(max(sm.qred[0], sm.qred[1]), max(sm.qred[2], sm.qred[3]));
            // exponents outside +-100 are left alone: such rows have scores of 0 or infinity
            const int e = mx == 0 ? 127 : min(max((int)(mx >> 7), 27), 227);
            const float s = __int_as_float((127 + 134 - e) << 23);
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                const int item = i * 128 + tid, row = item >> 3, j = item & 7;
                if (row >= R) break;
                uint32_t hi[4], lo[4];
                const uint32_t* w = reinterpret_cast<const uint32_t*>(x[i]);
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
                unsigned char* q = smem + C::kOffQ;
                const int rl = R + row;
                *reinterpret_cast<uint4*>(q + row * 128 + ((j ^ (row & 7)) << 4)) =
                    make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(q + rl * 128 + ((j ^ (rl & 7)) << 4)) =
                    make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            fence_async_shared();
            mbar_arrive(&sm.q_ready);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.raw_empty);
            return __int_as_float((127 - 134 + e) << 23);
        };

        dead |= !wait(&sm.seg_full[0], 0);
        if (!group_any(dead)) {
            seg = sm.segs[0];
            qc = convert(0, seg) * a.sm_scale * kLog2e;
            int g = 0;
            for (int k = 0;; ++k) {
                if (tid < R) sm.mref[tid] = kNoRef;
                sm.first_nan[tid] = INT32_MAX;
                float l[R];
#pragma unroll
                for (int r = 0; r < R; ++r) l[r] = 0.f;
                group_sync();
                const int lim_min = seg.lim0 + seg.row0 / group;
                const int32_t* lim = sm.lim[k & 1];
                bool stop = false;
                for (int t = seg.tile0; t < seg.tile1; ++t, ++g) {
                    const int b = g & 1, s = g % C::kStages;
                    const uint32_t ph = (uint32_t)(g / C::kStages) & 1;
                    dead |= !wait(&sm.meta_full[s], ph);
                    const float2 sc = sm.meta[s][tid / bs];
                    const int pos = t * kTileKeys + tid;
                    const bool in = pos < seg.keys;
                    const float c1 = in ? sc.x * qc : 0.f, c2 = c1 * 0.0625f;
                    const float lvs = in ? lg2(sc.y) : 0.f, inv = in ? __frcp_rn(sc.y) : 0.f;
                    const bool cut = (t + 1) * kTileKeys > lim_min;  // some row does not see all
                    dead |= !wait(&sm.s_full[b], (uint32_t)(g >> 1) & 1);
                    tc_fence_after();
                    // scores in base 2, with the value scale
                    float x[R];
                    {
                        constexpr int kC = R < 32 ? R : 32;
                        const float2 cc1 = make_float2(c1, c1), cc2 = make_float2(c2, c2);
                        const float2 lv = make_float2(lvs, lvs);
#pragma unroll
                        for (int q = 0; q < R; q += kC) {
                            uint32_t hi[kC], lo[kC];
                            if constexpr (R == 8) {
                                uint32_t both[16];
                                tmem_ld16(lanes + b * C::kNQ, both);
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    hi[i] = both[i];
                                    lo[i] = both[8 + i];
                                }
                            } else {
                                tmem_ld<kC>(lanes + b * C::kNQ + q, hi);
                                tmem_ld<kC>(lanes + b * C::kNQ + R + q, lo);
                            }
#pragma unroll
                            for (int i = 0; i < kC; i += 2) {
                                const float2 h2 = make_float2(__uint_as_float(hi[i]), __uint_as_float(hi[i + 1]));
                                const float2 l2 = make_float2(__uint_as_float(lo[i]), __uint_as_float(lo[i + 1]));
                                const float2 y = fma_f32x2(h2, cc1, fma_f32x2(l2, cc2, lv));
                                x[q + i] = y.x;
                                x[q + i + 1] = y.y;
                            }
                        }
                    }
                    if (cut) {
#pragma unroll
                        for (int r = 0; r < R; r += 4) {
                            const int4 m = *reinterpret_cast<const int4*>(lim + r);
                            x[r] = pos < m.x ? x[r] : -INFINITY;
                            x[r + 1] = pos < m.y ? x[r + 1] : -INFINITY;
                            x[r + 2] = pos < m.z ? x[r + 2] : -INFINITY;
                            x[r + 3] = pos < m.w ? x[r + 3] : -INFINITY;
                        }
                        // values: none beyond the context, no NaN where a row may not see it
                        dead |= !wait(&sm.v_full[s], ph);
                        unsigned char* row = smem + C::kOffV + s * kTileBytes + tid * kDim;
#pragma unroll 1
                        for (int j = 0; j < 8; ++j) {
                            uint4* p = reinterpret_cast<uint4*>(row + ((j ^ (tid & 7)) << 4));
                            if (!in) {
                                *p = make_uint4(0, 0, 0, 0);
                                continue;
                            }
                            uint4 v = *p;
                            uint32_t* w = reinterpret_cast<uint32_t*>(&v);
                            bool any = false;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t nan = __vcmpeq4(w[i] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                any |= nan != 0;
                                for (int y = 0; y < 4; ++y)
                                    if (nan >> (8 * y) & 1)
                                        atomicMin(&sm.first_nan[j * 16 + i * 4 + y], pos);
                                w[i] &= ~nan;
                            }
                            if (any) *p = v;
                        }
                    }
                    // does any score exceed its row's reference by too much?
                    float over = -INFINITY;
#pragma unroll
                    for (int r = 0; r < R; r += 4) {
                        const float4 m = *reinterpret_cast<const float4*>(sm.mref + r);
                        over = fmaxf(over, fmaxf(fmaxf(x[r] - m.x, x[r + 1] - m.y),
                                                 fmaxf(x[r + 2] - m.z, x[r + 3] - m.w)));
                    }
                    if (group_any(over > kPeak + kSlack || dead)) {
                        if (group_any(dead)) {  // a wait gave up: all four warps leave together
                            stop = true;
                            break;
                        }
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const int m = __reduce_max_sync(~0u, ordered(x[r]));
                            if (lane == (r & 31)) sm.red[warp][r] = unordered(m);
                        }
                        group_sync();
                        if (tid < R) {
                            const float m = fmaxf(fmaxf(sm.red[0][tid], sm.red[1][tid]),
                                                  fmaxf(sm.red[2][tid], sm.red[3][tid])) - kPeak;
                            const float old = sm.mref[tid], now = fmaxf(old, m);
                            sm.fac[tid] = ex2_approx(old - now);
                            sm.mref[tid] = now;
                        }
                        if (t > seg.tile0) {
                            dead |= !wait(&sm.pv_done[(g - 1) & 1], (uint32_t)((g - 1) >> 1) & 1);
                            tc_fence_after();
                        }
                        group_sync();
                        if (t > seg.tile0) {
#pragma unroll 1
                            for (int c = 0; c < 3 * R; c += 8) {  // R is a multiple of 8
                                uint32_t o[16];
                                // 16 columns are loaded and the first 8 stored with their factors
                                const int at = min(c, C::kNP - 16);
                                tmem_ld16(o_col + at, o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const int col = at + i;
                                    const float f = col >= c && col < c + 8 ? sm.fac[col % R] : 1.f;
                                    o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                }
                                tmem_st16(o_col + at, o);
                                tmem_st_wait();
                            }
                        }
#pragma unroll
                        for (int r = 0; r < R; ++r) l[r] *= sm.fac[r];
                    }
                    // weights, their sums, and three e4m3 terms of each
                    if (g >= 2) dead |= !wait(&sm.pv_done[b], (uint32_t)((g >> 1) - 1) & 1);
                    unsigned char* pt = smem + C::kOffP + b * C::kPBytes + tid * 128;
                    auto p_chunk = [&](int col) {  // 16 columns from col on, of this key's row
                        return reinterpret_cast<uint4*>(pt + (col >> 7) * 16384 +
                                                        ((((col & 127) >> 4) ^ (tid & 7)) << 4));
                    };
                    constexpr int kG = R < 16 ? R : 16;
                    const float2 inv2 = make_float2(inv, inv);
#pragma unroll
                    for (int q = 0; q < R; q += kG) {
                        uint32_t term[3][kG / 4];
#pragma unroll
                        for (int i = 0; i < kG; i += 2) {
                            const float2 m = *reinterpret_cast<const float2*>(sm.mref + q + i);
                            const float p0 = ex2_approx(x[q + i] - m.x), p1 = ex2_approx(x[q + i + 1] - m.y);
                            const float2 sum = fma_f32x2(make_float2(p0, p1), inv2,
                                                         make_float2(l[q + i], l[q + i + 1]));
                            l[q + i] = sum.x;
                            l[q + i + 1] = sum.y;
                            const __half2 p = __floats2half2_rn(p0, p1);
                            const uint16_t e0 = half2_to_e4m3(as_u32(p));
                            const __half2 r1 = __hmul2(__hsub2(p, as_half2(e4m3_to_half2(e0))),
                                                       __float2half2_rn(16.f));
                            const uint16_t e1 = half2_to_e4m3(as_u32(r1));
                            const __half2 r2 = __hmul2(__hsub2(r1, as_half2(e4m3_to_half2(e1))),
                                                       __float2half2_rn(32.f));
                            const uint16_t e2 = half2_to_e4m3(as_u32(r2));
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
                        if constexpr (R == 8) {
                            *p_chunk(0) = make_uint4(term[0][0], term[0][1], term[1][0], term[1][1]);
                            *p_chunk(16) = make_uint4(term[2][0], term[2][1], 0, 0);
                        } else {
#pragma unroll
                            for (int c = 0; c < 3; ++c)
                                *p_chunk(c * R + q) = make_uint4(term[c][0], term[c][1], term[c][2], term[c][3]);
                        }
                    }
                    fence_async_shared();
                    tc_fence_before();
                    mbar_arrive(&sm.p_ready[b]);
                }
                if (stop) break;
                // the next segment's q, so that its first scores run under this one's outputs
                const int kn = k + 1;
                dead |= !wait(&sm.seg_full[kn % kSegs], (uint32_t)(kn / kSegs) & 1);
                if (group_any(dead)) break;
                const Seg next = sm.segs[kn % kSegs];
                float qc_next = 0.f;
                if (next.n >= 0) qc_next = convert(kn, next) * a.sm_scale * kLog2e;
                // outputs: thread = channel
                const bool some = seg.tile1 > seg.tile0;
                if (some) {
                    dead |= !wait(&sm.pv_done[(g - 1) & 1], (uint32_t)((g - 1) >> 1) & 1);
                    tc_fence_after();
                    warp_sums<R>(l, lane);
                    if (lane < R) sm.red[warp][lane] = l[0];
                    if constexpr (R == 64) sm.red[warp][32 + lane] = l[32];
                    group_sync();
                    if (tid < R) {
                        const float sum = sm.red[0][tid] + sm.red[1][tid] + sm.red[2][tid] + sm.red[3][tid];
                        if (seg.slot >= 0) {
                            parts[seg.slot].m[tid] = sm.mref[tid];
                            parts[seg.slot].l[tid] = sum;
                            sm.fac[tid] = 1.f;
                        } else {
                            sm.fac[tid] = sum == 0.f ? 0.f : 1.f / sum;
                        }
                    }
                    group_sync();
                }
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
                const int32_t* orow = sm.orow[k & 1];
                const int nan_from = sm.first_nan[tid];
#pragma unroll 1
                for (int q = 0; q < seg.rows; q += 8) {
                    float o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = 0.f;
                    if (some) {
#pragma unroll
                        for (int c = 2; c >= 0; --c) {  // small terms first
                            uint32_t u[16];
                            const int col = c * R + q, at = min(col, C::kNP - 16);
                            tmem_ld16(o_col + at, u);
                            const float w = c == 0 ? 1.f : c == 1 ? 0x1p-4f : 0x1p-9f;
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                o[i] += w * __uint_as_float(col == at ? u[i] : u[8 + i]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (q + i >= seg.rows) break;
                        const float y = lim[q + i] > nan_from ? NAN : some ? o[i] * sm.fac[q + i] : 0.f;
                        if (seg.slot >= 0) parts[seg.slot].o[q + i][tid] = y;
                        else out[(int64_t)orow[q + i] * kDim + tid] = __float2bfloat16_rn(y);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.seg_empty[k % kSegs]);
                if (next.n < 0) break;
                group_sync();  // mref, fac and the sums are free again
                seg = next;
                qc = qc_next;
            }
        }
        if (dead) sm.abort_flag = 1;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 5) tmem_dealloc(tmem, C::kTmem);
}

// Joins the partial results of the unit that CTA blockIdx.x began and others went on with: a warp
// per row, four channels a lane, in key order.
template <int R>
__global__ void __launch_bounds__(128) paged_attention_join_kernel(const AttnArgs a, int ctas) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PartDesc* descs = static_cast<const PartDesc*>(a.workspace);
    const Part<R>* parts = reinterpret_cast<const Part<R>*>(static_cast<const char*>(a.workspace) +
                                                            (size_t)ctas * 2 * sizeof(PartDesc));
    const int c = blockIdx.x, lane = threadIdx.x & 31, row = blockIdx.y * 4 + (threadIdx.x >> 5);
    const PartDesc d = descs[2 * c + 1];
    if (!d.valid) return;
    const Run r = load_run(a, d.n, nullptr);
    const int group = a.heads / a.kv_heads, at = d.rt * R + row;
    if (at >= r.len * group) return;
    int last = c + 1;
    while (last < ctas - 1 && !(descs[2 * last].valid && descs[2 * last].ends)) ++last;
    auto slot_of = [&](int i) { return i == c ? 2 * c + 1 : 2 * i; };
    float m = kNoRef;
    for (int i = c; i <= last; ++i) m = fmaxf(m, parts[slot_of(i)].m[row]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 4
    for (int i = c; i <= last; ++i) {
        const Part<R>& p = parts[slot_of(i)];
        const float f = ex2_approx(p.m[row] - m);
        const float4 x = *reinterpret_cast<const float4*>(&p.o[row][lane * 4]);
        l += f * p.l[row];
        o.x += f * x.x;
        o.y += f * x.y;
        o.z += f * x.z;
        o.w += f * x.w;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t out_row = (int64_t)(r.q0 + at / group) * a.heads + d.head * group + at % group;
    uint2 y = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + out_row * kDim + lane * 4) = y;
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
    cudaError_t e = cudaFuncSetAttribute(paged_attention_kernel<R>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem_bytes<R>());
    if (e != cudaSuccess) return e;
    paged_attention_kernel<R><<<ctas_of<R>(), kAttnThreads, smem_bytes<R>(), stream>>>(a, km, vm, status);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas_of<R>(), R / 4);
    cfg.blockDim = dim3(128);
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
