// kda_paged_attn.cuh — what the two paged attention kernels share: the list of work and its equal
// shares, the producer of the cache's tiles, the conversion of values, and the joining of partial
// results.  A kernel is parametrised by R, the rows of one key head that it takes at a time.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include "kda_common.cuh"
#include "kda_paged.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace attn {

using namespace sm100;

constexpr int kTileKeys = 128;
constexpr int kTileBytes = kTileKeys * kDim;  // one K or V tile, e4m3
constexpr int kSegs = 4, kMetas = 4;          // work descriptors, tiles' page scales in flight
constexpr int kMaxTilePages = 8;              // pages of 16 tokens in a tile
// Units this short, and cuts this near to a unit's end, are not cut, so that short calls need no
// joining: one token over 257 takes 10.9 us, 12.3 where units of two tiles are cut.  With units of 8
// and cuts within 4 tiles prefill chunks gain (338 -> 333 us) and decode batches lose (111.5 -> 114).
constexpr int kSnapUnit = 4, kSnapEdge = 2;
constexpr int kGrainTiles = 4;                // least share of a CTA (the same token: 8 16.1 us, 2 no change)
constexpr long long kAttnWaitLimit = 4000000000LL;  // clock cycles (about 2 s)
constexpr float kNoRef = -1e37f;              // reference of a row that has seen no key
constexpr float kLog2e = 1.4426950408889634f;

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

// Barriers and rings between the producer, the issuer and the other warps.
template <int kKStages, int kVStages, int kThreads>
struct Ring {
    float4 meta[kMetas][kMaxTilePages];  // a tile's pages: key scale, log2 and inverse of value scale
    Seg segs[kSegs];
    int32_t first_nan[kSegs][kDim];      // per channel: first key whose value is NaN, where masked
    uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
    uint64_t meta_full[kMetas], meta_empty[kMetas], seg_full[kSegs], seg_empty[kSegs];
    uint64_t val_full[2], raw_full, raw_empty;
    // the CTA's share: (request, head, row tile, tile) and place of its ends
    int64_t scan[kThreads / 32];
    int64_t pos[2];
    int32_t at[2][4];
    uint32_t tmem;
    int32_t abort_flag;

    // v_readers, meta_readers, seg_readers: arrivals that free a value tile, page scales, a segment
    __device__ __forceinline__ void init(int v_readers, int meta_readers, int seg_readers,
                                         int val_writers, int raw_readers) {
        for (int s = 0; s < kKStages; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 1);
        }
        for (int s = 0; s < kVStages; ++s) {
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], v_readers);
        }
        for (int s = 0; s < kMetas; ++s) {
            mbar_init(&meta_full[s], 1);
            mbar_init(&meta_empty[s], meta_readers);
        }
        for (int s = 0; s < kSegs; ++s) {
            mbar_init(&seg_full[s], 1);
            mbar_init(&seg_empty[s], seg_readers);
        }
        for (int b = 0; b < 2; ++b) mbar_init(&val_full[b], val_writers);
        mbar_init(&raw_full, 1);
        mbar_init(&raw_empty, raw_readers);
        abort_flag = 0;
    }
};

// Workspace: per CTA two partial results (the unit it begins in, the unit it ends in).
struct PartDesc {
    int32_t valid, ends;              // ends: the unit's last part
    int32_t q0, head, row0, rows;     // as in Seg
    int32_t pad[2];
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
    // By a whole warp, with one answer for all of it.
    __device__ __forceinline__ bool warp(uint64_t* bar, uint32_t parity) const {
        return __all_sync(~0u, (*this)(bar, parity));
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
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
    return p != 0;
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
__device__ __forceinline__ uint16_t float2_to_e5m2(float lo, float hi) {
    uint16_t c;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
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
template <int R, int kThreads, class Sm>
__device__ __forceinline__ void find_share(const AttnArgs& a, Sm& sm, int* status) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, N = a.num_seqs;
    const int group = a.heads / a.kv_heads;
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

// ------------------------------------------------------------------------------- warp roles
// The producer warp: walks the share, hands out segments and fills the rings.  kRaw: the rows of q
// go to shared memory at off_raw; else they are only fetched into L2.
template <int R, int kKStages, int kVStages, bool kRaw, class Sm>
__device__ __forceinline__ void produce(const AttnArgs& a, Sm& sm, unsigned char* smem,
                                        uint32_t off_k, uint32_t off_v, uint32_t off_raw,
                                        const CUtensorMap& k_map, const CUtensorMap& v_map,
                                        PartDesc* descs, const Waiter& wait, int* status) {
    const int lane = threadIdx.x & 31, group = a.heads / a.kv_heads, bs = a.page_size;
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
        if (k >= kSegs) ok = wait.warp(&sm.seg_empty[sk], (k / kSegs - 1) & 1);
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
                const PartDesc d = {1, t1 == u, r.q0, h, row0, rows, {0, 0}};
                descs[slot] = d;
            }
        }
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
        if constexpr (kRaw) {  // its rows of q, token by token
            if (k >= 1) ok = wait.warp(&sm.raw_empty, (k - 1) & 1);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&sm.raw_full, (uint32_t)rows * 256);
            __syncwarp();
            for (int tk = row0 / group + lane; tk * group < row0 + rows; tk += 32) {
                const int ra = max(row0, tk * group), rb = min(row0 + rows, (tk + 1) * group);
                bulk_load(smem + off_raw + (ra - row0) * 256,
                          q + (int64_t)(r.q0 + tk) * a.q_stride + (h * group + ra - tk * group) * kDim,
                          (uint32_t)(rb - ra) * 256, &sm.raw_full);
            }
        } else {  // its rows of q into L2, for the threads that read them
            for (int row = lane; row < 2 * rows; row += 32) {
                const int at = row0 + (row >> 1);
                const __nv_bfloat16* p = q + (int64_t)(r.q0 + at / group) * a.q_stride +
                                         (h * group + at % group) * kDim + (row & 1) * 64;
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
            }
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
                float2 s = make_float2(0.f, 0.f);  // of a page without keys: no score, no weight
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
                const int sk = g % kKStages, sv = g % kVStages, me = g % kMetas;
                const int live = min(pp, pages - t * pp);  // pages of this tile with keys
                next = checked(next);
                const float2 sc_next = scales_of(next);
                const int after = page_of(t + 2);
                if (g >= kKStages) ok = wait.warp(&sm.k_empty[sk], (uint32_t)(g / kKStages - 1) & 1);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&sm.k_full[sk], (uint32_t)(live * bs * kDim));
                __syncwarp();
                if (lane < live)
                    tma_load_3d(smem + off_k + sk * kTileBytes + lane * bs * kDim, &k_map,
                                &sm.k_full[sk], 0, h * bs, id);
                if (g >= kMetas) ok = wait.warp(&sm.meta_empty[me], (uint32_t)(g / kMetas - 1) & 1);
                if (!ok) break;
                if (lane < kMaxTilePages)
                    sm.meta[me][lane] = make_float4(sc.x, lane < live ? lg2(sc.y) : 0.f,
                                                    lane < live ? rcp(sc.y) : 0.f, 0.f);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.meta_full[me]);
                if (g >= kVStages) ok = wait.warp(&sm.v_empty[sv], (uint32_t)(g / kVStages - 1) & 1);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&sm.v_full[sv], (uint32_t)(live * bs * kDim));
                __syncwarp();
                if (lane < live)
                    tma_load_3d(smem + off_v + sv * kTileBytes + lane * bs * kDim, &v_map,
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
        if (k >= kSegs) ok = wait.warp(&sm.seg_empty[sk], (k / kSegs - 1) & 1);
        if (ok && lane == 0) {
            sm.segs[sk].n = -1;
            mbar_arrive(&sm.seg_full[sk]);
        }
    }
    // every copy has landed before the CTA may end: the consumers waited for them all, unless
    // a wait gave up
    if (*static_cast<volatile int32_t*>(&sm.abort_flag)) {
        for (int i = max(0, g - kKStages); i <= g; ++i)
            mbar_wait(&sm.k_full[i % kKStages], (uint32_t)(i / kKStages) & 1, kAttnWaitLimit / 8);
        for (int i = max(0, g - kVStages); i <= g; ++i)
            mbar_wait(&sm.v_full[i % kVStages], (uint32_t)(i / kVStages) & 1, kAttnWaitLimit / 8);
        if (kRaw && k > 0) mbar_wait(&sm.raw_full, (k - 1) & 1, kAttnWaitLimit / 8);
    }
}

// The four warps that convert values: e4m3 tiles into f16 ones (two column halves of 128 keys x 128
// bytes), one key's row a thread.  val_empty[b] completes when buffer b has been read.
// begin(k, seg) runs at the start of segment k and says whether its waits ended.
template <int kVStages, class Sm, class Begin>
__device__ __forceinline__ void convert_values(Sm& sm, unsigned char* smem, uint32_t off_v,
                                               uint32_t off_val, uint64_t* val_empty, int key,
                                               int group, const Waiter& wait, Begin begin) {
    const int lane = key & 31;
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
        ok &= begin(k, seg);
        for (; t < tile1; ++t, ++g) {
            const int b = g & 1, s = g % kVStages;
            if (!(ok = wait(&sm.v_full[s], (uint32_t)(g / kVStages) & 1))) break;
            if (g >= 2 && !(ok = wait(&val_empty[b], (uint32_t)((g >> 1) - 1) & 1))) break;
            const unsigned char* row = smem + off_v + s * kTileBytes + key * kDim;
            unsigned char* to = smem + off_val + b * 2 * kTileBytes + key * 128;
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
}

// Joins the partial results of the units that more than one CTA worked on, in key order.  Unit u's
// parts are the last of the CTA that began it and the first of those that went on.  Every block
// lists the units (the descriptors are few) and takes its share of the items: a row a warp of a
// unit in up to kJoinParts parts (four rows a warp of a large tile in two), else one row whose parts
// the eight warps share.  Nothing an item loads depends on another load of it, so an item takes one
// trip to memory.  What it adds to a call
// is mostly its launch and three trips (descriptors, parts, outputs): 6 us for 64 decode requests, 7
// for 128 windows, 10 for 64 rows in 152 parts, 11 for 150 units of 256 rows in two.  Eight rows of
// parts in flight instead of four, and one CTA a unit (12 to 86 us), gained nothing.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32, kJoinParts = 16;
constexpr int kJoinBlocks = 4 * kPlanSMs;
template <int R>
__global__ void __launch_bounds__(kJoinThreads, 4) paged_attention_join_kernel(const AttnArgs a, int ctas) {
    constexpr int kMaxCtas = 2 * kPlanSMs, kPer = (kMaxCtas + kJoinThreads - 1) / kJoinThreads;
    __shared__ uint32_t ends[kPer * kJoinWarps];  // CTAs whose first part ends its unit
    __shared__ int32_t first_item[kMaxCtas + 1], sums[kJoinWarps];
    __shared__ float part_m[kJoinWarps], part_l[kJoinWarps];
    __shared__ float4 part_o[kJoinWarps][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = a.heads / a.kv_heads;
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
            end |= d.x && d.y;
            begins[i] = descs[2 * c + 1].valid;
            any |= begins[i];
        }
        const uint32_t m = __ballot_sync(~0u, end);
        if (lane == 0) ends[i * kJoinWarps + warp] = m;
    }
    if (!__syncthreads_or(any)) return;
    auto last_of = [&](int c) {  // the CTA in whose share the unit that c began ends
        int w = (c + 1) >> 5;
        uint32_t bits = ends[w] & (~0u << ((c + 1) & 31));
        while (bits == 0) bits = ends[++w];
        return w * 32 + __ffs(bits) - 1;
    };
    // items before each unit: a scan over the CTAs
    int items = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int c = i * kJoinThreads + tid;
        int mine = 0;
        if (begins[i]) {
            const int count = last_of(c) - c + 1;
            mine = R >= 32 && count == 2 ? R / 32 : count <= kJoinParts ? (R + kJoinWarps - 1) / kJoinWarps : R;
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
        const int last = last_of(c), count = last - c + 1, at = item - first_item[c];
        const bool shared = count > kJoinParts;
        const int row = shared ? at : at * kJoinWarps + warp;
        const PartDesc d = descs[2 * c + 1];
        auto give = [&](int row, float4 o, float l) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const int r = d.row0 + row;
            const int64_t to = (int64_t)(d.q0 + r / group) * a.heads + d.head * group + r % group;
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + to * kDim + lane * 4) =
                make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        };
        if (R >= 32 && count == 2) {  // the usual case of large tiles: four rows a warp
            const Part<R>& p = parts[2 * c + 1];
            const Part<R>& q = parts[2 * c + 2];
            const int r0 = at * 32 + warp * 4;
            float4 x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = *reinterpret_cast<const float4*>(&p.o[r0 + i][lane * 4]);
                y[i] = *reinterpret_cast<const float4*>(&q.o[r0 + i][lane * 4]);
            }
            const float4 pm = *reinterpret_cast<const float4*>(&p.m[r0]), qm = *reinterpret_cast<const float4*>(&q.m[r0]);
            const float4 pl = *reinterpret_cast<const float4*>(&p.l[r0]), ql = *reinterpret_cast<const float4*>(&q.l[r0]);
            const float ms[2][4] = {{pm.x, pm.y, pm.z, pm.w}, {qm.x, qm.y, qm.z, qm.w}};
            const float ls[2][4] = {{pl.x, pl.y, pl.z, pl.w}, {ql.x, ql.y, ql.z, ql.w}};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float m = fmaxf(ms[0][i], ms[1][i]), u = ex2_approx(ms[0][i] - m), w = ex2_approx(ms[1][i] - m);
                if (r0 + i < d.rows)
                    give(r0 + i, make_float4(u * x[i].x + w * y[i].x, u * x[i].y + w * y[i].y,
                                             u * x[i].z + w * y[i].z, u * x[i].w + w * y[i].w),
                         u * ls[0][i] + w * ls[1][i]);
            }
            continue;
        }
        auto part = [&](int i) -> const Part<R>& { return parts[i == 0 ? 2 * c + 1 : 2 * (c + i)]; };
        // this warp's parts: all, or every kJoinWarps-th
        const int step = shared ? kJoinWarps : 1, from = shared ? warp : 0;
        const int mine = (count - from + step - 1) / step;
        float m = kNoRef, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = 0; i0 < mine; i0 += 32) {
            // 32 parts' references and sums, then their rows four at a time, all independent
            const int i = min(i0 + lane, mine - 1), n = min(mine - i0, 32);
            const Part<R>& p = part(from + i * step);
            const float pm = p.m[row], pl = lane < n ? p.l[row] : 0.f;
            float4 y[4];
            auto fetch = [&](int j) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    y[x] = *reinterpret_cast<const float4*>(
                        &part(from + (i0 + min(j + x, n - 1)) * step).o[row][lane * 4]);
            };
            fetch(0);
            float top = pm;
#pragma unroll
            for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
            top = fmaxf(top, m);
            const float keep = ex2_approx(m - top), f = lane < n ? ex2_approx(pm - top) : 0.f;
            m = top;
            l = l * keep;
            o.x *= keep;
            o.y *= keep;
            o.z *= keep;
            o.w *= keep;
            float fl = f * pl;
#pragma unroll
            for (int x = 16; x; x >>= 1) fl += __shfl_xor_sync(~0u, fl, x);
            l += fl;
            for (int j = 0; j < n; j += 4) {
                if (j > 0) fetch(j);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if (j + x >= n) break;
                    const float w = __shfl_sync(~0u, f, j + x);
                    o.x += w * y[x].x;
                    o.y += w * y[x].y;
                    o.z += w * y[x].z;
                    o.w += w * y[x].w;
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
                for (int j = 0; j < kJoinWarps; ++j) m = fmaxf(m, part_m[j]);
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
        if (row < d.rows && (!shared || warp == 0)) give(row, o, l);
    }
}

// ---------------------------------------------------------------------------------------- host
template <int R>
constexpr size_t workspace_of(int ctas) { return (size_t)ctas * 2 * (sizeof(PartDesc) + sizeof(Part<R>)); }

template <int R>
cudaError_t launch_join(const AttnArgs& a, int ctas, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kJoinBlocks);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_attention_join_kernel<R>, a, ctas);
}

}  // namespace attn

// Row tiles of 64, 128 and 256 rows (kda_paged_attn_wide.cu).
size_t paged_attention_wide_workspace(int rows);
cudaError_t launch_paged_attention_wide(int rows, const AttnArgs& a, const CUtensorMap& k_map,
                                        const CUtensorMap& v_map, bool join, int* status,
                                        cudaStream_t stream);

}  // namespace kda
