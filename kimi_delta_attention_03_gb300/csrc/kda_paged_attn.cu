// kda_paged_attn.cu — attention over a paged cache held in e4m3 with a scale per (page, head).
//
// For row (token i of a run of L, query head h) of a request with context c, over keys
// j = 0 .. c - L + i of key head h / G (G = H / Hkv query heads share one):
//     z_j = (q . k_j) s_k(page of j) sm_scale,   o = sum_j e^(z_j - m) v_j s_v / sum_j e^(z_j - m)
//
// The cache's bytes go from HBM to the tensor cores as they are: the products take the e4m3 tiles
// that TMA puts into shared memory as tcgen05 operands (kind::f8f6f4), 128 keys at a time.  What
// meets them is split into 8-bit terms:
//   S^T [128 keys x R] = K [128 x 128] (Q_hi + Q_lo)^T    q = (Q_hi + Q_lo) / s: a bf16 has 8
//                        significant bits; 4 in e4m3 leave at most +-8 units, which e5m2's 3 hold.  s
//                        is a power of two of each row's own, so a row does not depend on the size of
//                        its neighbours; elements below 2^-13 of a row's largest are held within 2^-21
//                        of it
//   O^T [128 channels x 3R] += V^T [128 x 128] [P_0 P_1 P_2]    p = P_0 + P_1 / 2^5 + P_2 / 2^10: a
//                        term's scale is the largest that keeps what the one before left of p <= 2^8
//                        within e4m3.  All 11 bits of an f16 p down to 2^-15 of a row's largest weight,
//                        within 2^-25 of it below, where P_2 ends.  There each key of a tile rounds from
//                        a place of its own in P_2's last step, so that the errors of equal weights,
//                        which would add up over a long light tail, cancel to 2^-29 over 128 keys.
// R (8, 16 or 32) rows of one key head are a tile's columns, so a few rows cost few columns, and the
// terms of weights are extra columns, not extra passes over V.  (Q_lo as columns of its own, in e4m3
// and scaled by 2^4, costs the softmax warps a load and an addition a score: 64 requests of 16 rows
// a head over 512 .. 16K tokens, 615 MB of cache, take 130 us so and 120 as they are.)  At R = 32 the
// splitting of weights, which grows with the rows, would cost more than it saves: there weights are
// one f16 number (11 bits), and four more warps widen the values to f16 (kind::f16) once per tile.
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
//        are formed against a reference that a row's scores may exceed by up to 2^2 before the
//        four warps agree (one barrier with a vote) to raise it and rescale their columns of O^T,
//        which after the first tile is rare.
//   producer: work list, page tables and scales a tile ahead, TMA of K, V and raw q
//   issuer of the MMAs: scores of tile j + 1 before the weighted sum of tile j
//
// What bounds it: HBM.  64 decode requests over 512 .. 16K tokens of 8 key heads (615 MB of cache)
// take 111.5 us, 82% of the measured copy bandwidth (5.5 TB/s); the rest is the ends: the share, the
// first tiles' latency, the last outputs and the joining of cut units (6 us of it).  Two CTAs
// to an SM fill each other's waits.  Two key and three value stages in the ring: a value tile is held
// until its weighted sum is done (two and two: 115.5 us; three and two: 115.8).  One request of one
// token is latency: 10.9 us for three dependent tiles.
//
// Masked places.  Keys beyond a row's limit get weight 0.  Values beyond the request's context are
// zeroed in shared memory (0 * NaN), and a NaN value inside it is replaced by 0 in tiles where some
// row may not see it and put back into the rows that do.
#include <algorithm>
#include <atomic>
#include <mutex>

#include "kda_paged_attn.cuh"

namespace kda {
namespace {

using namespace attn;

template <int R>
struct Cfg {
    static constexpr bool kHalf = R >= 32;                  // weights and values meet in f16
    static constexpr int kRW = R == 8 ? 8 : 16;  // rows of a softmax warpgroup
    static constexpr int kGroups = R / kRW;                 // softmax warpgroups
    static constexpr int kSoft = kGroups * 128;             // their threads
    static constexpr int kConv = kHalf ? 128 : 0;           // threads that convert values
    static constexpr int kThreads = kSoft + kConv + 64;     // and the producer's and the issuer's
    static constexpr int kTerms = kHalf ? 1 : 3;            // numbers a weight is held in
    static constexpr int kNQ = R < 16 ? 16 : R;             // columns of a score tile (at least 16)
    static constexpr int kNP = (kTerms * R + 15) / 16 * 16; // columns of the output tile
    static constexpr int kCtasPerSm = R <= 16 ? 2 : 1;
    static constexpr int kKStages = R <= 16 ? 2 : 3;
    // (a value tile is held longer than a key tile: until its weighted sum is done)
    static constexpr int kVStages = 3;
    static constexpr int kTmem = R == 8 ? 64 : 128;
    // weights: a row of 128 bytes for each of 128 keys, two buffers, side by side where both fit
    static constexpr bool kPHalves = R <= 16;
    static constexpr int kPBytes = kPHalves ? 64 : 16384;
    static constexpr int kValBytes = kHalf ? 2 * kTileBytes : 0;  // a tile of values in f16
    // weights are 2^kPeak at their row's reference and may reach 2^(kPeak + kSlack): below f16's
    // largest, 65504, or 2^8, where what P_0 leaves is up to 8 and 2^5 times that within e4m3
    static constexpr float kPeak = kHalf ? 4.f : 6.f, kSlack = kHalf ? 11.5f : 2.f;
    static constexpr uint32_t kOffK = 0;
    static constexpr uint32_t kOffV = kOffK + kKStages * kTileBytes;
    static constexpr uint32_t kOffVal = kOffV + kVStages * kTileBytes;
    static constexpr uint32_t kOffP = kOffVal + 2 * kValBytes;
    static constexpr uint32_t kOffQ = kOffP + (kPHalves ? 1 : 2) * 16384;
    static constexpr uint32_t kOffRaw = kOffQ + 2 * kNQ * 128;
    static constexpr uint32_t kOffSmall = kOffRaw + R * 256;
    static_assert(2 * kNQ + kNP <= kTmem, "tensor memory columns");
    static_assert(kTerms * R * (kHalf ? 2 : 1) <= (kPHalves ? 64 : 128), "a key's weights and their row");
};

template <int R>
struct Small : Ring<Cfg<R>::kKStages, Cfg<R>::kVStages, Cfg<R>::kThreads> {
    alignas(16) float mref[R];
    alignas(16) float qs[2][R];  // score scale of each row: sm_scale log2 e / s
    float fac[R];
    int32_t lim[2][R];
    int32_t orow[2][R];
    float red[4][R];
    uint64_t s_full[2], p_ready[2], pv_done[2], q_ready, q_taken;
};

template <int R>
constexpr size_t smem_bytes() { return Cfg<R>::kOffSmall + sizeof(Small<R>) + 1024; }
static_assert(smem_bytes<32>() <= 232448, "shared memory of a CTA");
static_assert(smem_bytes<16>() <= 115712 && smem_bytes<8>() <= 115712, "shared memory of two CTAs");

// ------------------------------------------------------------------------------ small wrappers
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
// Order-preserving map of floats to integers (for an integer maximum over a warp).
__device__ __forceinline__ int32_t ordered(float x) {
    const int32_t i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int32_t i) {
    return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
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
    find_share<R, C::kThreads>(a, sm, status);
    if (tid < 2) {  // partial results of this CTA: none so far
        PartDesc d = {};
        descs[2 * blockIdx.x + tid] = d;
    }
    if (sm.pos[0] >= sm.pos[1]) return;  // the same for every thread

    if (tid == 0) {
        sm.init(C::kHalf ? C::kConv / 32 : 1, C::kSoft / 32, (C::kSoft + C::kConv) / 32 + 1,
                C::kHalf ? C::kConv : 1, C::kSoft / 32);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm.s_full[b], 1);
            mbar_init(&sm.p_ready[b], C::kSoft);
            mbar_init(&sm.pv_done[b], 1);
        }
        mbar_init(&sm.q_ready, C::kSoft);
        mbar_init(&sm.q_taken, 1);
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
        produce<R, C::kKStages, C::kVStages, true>(a, sm, smem, C::kOffK, C::kOffV, C::kOffRaw, k_map,
                                                   v_map, descs, wait, status);
    } else if (warp == kIssuer) {
        // ------------------------------------------------------------------------ MMA issuer
        // The whole warp walks the work, one elected lane issues: descriptors in uniform registers.
        {
            constexpr uint32_t kIdHi = idesc_zero(C::kNQ, false, false);
            constexpr uint32_t kIdLo = kIdHi | 1u << 10;  // the second operand in e5m2
            constexpr uint32_t kIdP = idesc_zero(C::kNP, true, true);  // f16's code is e4m3's: 0
            const uint32_t base = __shfl_sync(~0u, saddr(smem), 0), tm = __shfl_sync(~0u, tmem, 0);
            const uint32_t o_col = tm + 2 * C::kNQ;
            const uint64_t q_desc = smem_desc(base + C::kOffQ, 16, 1024);
            auto scores = [&](int g) {
                const int s = g % C::kKStages;
                if (!wait.warp(&sm.k_full[s], (uint32_t)(g / C::kKStages) & 1)) return false;
                tc_fence_after();
                const uint64_t k_desc = smem_desc(base + C::kOffK + s * kTileBytes, 16, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)  // 32 channels (32 bytes of a swizzled row) each
                        mma_f8(tm + (g & 1) * C::kNQ, k_desc + 2 * (i & 3),
                               q_desc + (i >> 2) * (C::kNQ * 128 >> 4) + 2 * (i & 3), i < 4 ? kIdHi : kIdLo, i > 0);
                    mma_commit(&sm.k_empty[s]);
                    mma_commit(&sm.s_full[g & 1]);
                }
                __syncwarp();
                return true;
            };
            auto sums = [&](int g, bool first) {
                const int b = g & 1, s = g % C::kVStages;
                bool ok = C::kHalf ? wait(&sm.val_full[b], (uint32_t)(g >> 1) & 1)
                                   : wait(&sm.v_full[s], (uint32_t)(g / C::kVStages) & 1);
                ok &= wait(&sm.p_ready[b], (uint32_t)(g >> 1) & 1);
                if (!__all_sync(~0u, ok)) return false;  // the lanes leave together
                tc_fence_after();
                const uint64_t p_desc = smem_desc(base + C::kOffP + b * C::kPBytes, 16384, 1024);
                const uint64_t v_desc = C::kHalf ? smem_desc(base + C::kOffVal + b * C::kValBytes, 16384, 1024)
                                                 : smem_desc(base + C::kOffV + s * kTileBytes, 16384, 1024);
                if (elect_one()) {
                    if constexpr (C::kHalf) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)  // 16 keys (16 rows of 128 bytes) each
                            mma_ss(o_col, v_desc + 128 * i, p_desc + 128 * i, kIdP, !first || i > 0);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)  // 32 keys (32 rows of 128 bytes) each
                            mma_f8(o_col, v_desc + 256 * i, p_desc + 256 * i, kIdP, !first || i > 0);
                        mma_commit(&sm.v_empty[s]);
                    }
                    mma_commit(&sm.pv_done[b]);
                }
                __syncwarp();
                return true;
            };
            int g = 0, before = 0;  // tiles so far; tiles of the last segment, whose last is open
            for (int k = 0;; ++k) {
                if (!wait.warp(&sm.seg_full[k % kSegs], (uint32_t)(k / kSegs) & 1)) break;
                const Seg& seg = sm.segs[k % kSegs];
                const int n = __shfl_sync(~0u, seg.n, 0), tiles = __shfl_sync(~0u, seg.tile1 - seg.tile0, 0);
                if (before > 0 && !sums(g - 1, before == 1)) break;
                before = 0;
                if (n < 0) break;
                if (lane == 0) mbar_arrive(&sm.seg_empty[k % kSegs]);
                __syncwarp();
                if (!wait.warp(&sm.q_ready, k & 1)) break;
                if (lane == 0) mbar_arrive(&sm.q_taken);
                __syncwarp();
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
        convert_values<C::kVStages>(sm, smem, C::kOffV, C::kOffVal, sm.pv_done, tid - C::kSoft, group, wait,
                                    [](int, const Seg&) { return true; });
    } else {
        // --------------------------------------------------------- scores, weights and outputs
        // Warpgroup wg has rows r0 .. r0 + kRW - 1 of the tile; its thread `key` has one key of the
        // tile (a TMEM lane) for the weights and one channel for the outputs.
        constexpr int kRW = C::kRW;
        const int wg = warp >> 2, key = tid & 127, r0 = wg * kRW;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // TMEM lane 32 * (warp % 4)
        const uint32_t o_col = lanes + 2 * C::kNQ + r0;
        const int page_at = key / bs;
        // where this key rounds in the last term's smallest step, 2^-9: the 128 keys of a tile evenly
        // over 15/16 of it (so that what the term holds exactly stays), neighbours far apart
        const __half2 place = __float2half2_rn((float)((2 * (int)(__brev(key) >> 25) - 127) * 15) * 0x1p-21f);
        bool dead = false;  // a wait gave up: run on to where all warpgroups can leave together

        // Rows of q of segment k as an e4m3 and an e5m2 term, each row scaled by a power of two s so that its
        // largest lies in [128, 256): eight threads a row, an item is 16 channels.
        constexpr int kItems = (R * 8 + C::kSoft - 1) / C::kSoft;
        auto convert = [&](int k, const Seg& sg) {
            dead |= !wait(&sm.raw_full, k & 1);
            // Not a second phase of q_ready before the issuer has seen the first: a segment without
            // tiles makes nothing else wait for it.
            if (k > 0) dead |= !wait(&sm.q_taken, (k - 1) & 1);
            if (tid < R) {
                const int at = sg.row0 + tid, tok = at / group;
                sm.lim[k & 1][tid] = tid < sg.rows ? sg.lim0 + tok : 0;
                sm.orow[k & 1][tid] = (sg.q0 + tok) * a.heads + sg.head * group + at % group;
            }
#pragma unroll
            for (int it = 0; it < kItems; ++it) {
                const int row = (it * C::kSoft + tid) >> 3, j = tid & 7;
                uint4 x[2] = {};
                if (row < sg.rows) {
                    const uint4* p = reinterpret_cast<const uint4*>(smem + C::kOffRaw + row * 256 + j * 32);
                    x[0] = p[0];
                    x[1] = p[1];
                }
                const uint32_t* w = reinterpret_cast<const uint32_t*>(x);
                uint32_t mx = 0;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint32_t lo = w[c] & 0x7fffu, hi = (w[c] >> 16) & 0x7fffu;
                    mx = max(mx, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
                }
#pragma unroll
                for (int d = 1; d < 8; d <<= 1) mx = max(mx, __shfl_xor_sync(~0u, mx, d));
                const int e = max((int)(mx >> 7), 8);  // below 2^-119 the scale stays what it is there
                const float s = __int_as_float((127 + 134 - e) << 23);
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    float y0 = __uint_as_float(w[c] << 16) * s, y1 = __uint_as_float(w[c] & 0xffff0000u) * s;
                    if (isinf(y0)) y0 = NAN;
                    if (isinf(y1)) y1 = NAN;
                    const uint16_t h2 = float2_to_e4m3(y0, y1);
                    const float2 b = __half22float2(as_half2(e4m3_to_half2(h2)));
                    const uint16_t l2 = float2_to_e5m2(y0 - b.x, y1 - b.y);
                    if (c & 1) {
                        hi[c >> 1] |= (uint32_t)h2 << 16;
                        lo[c >> 1] |= (uint32_t)l2 << 16;
                    } else {
                        hi[c >> 1] = h2;
                        lo[c >> 1] = l2;
                    }
                }
                if (row < R) {
                    if (j == 0)
                        sm.qs[k & 1][row] = __int_as_float((127 - 134 + e) << 23) * a.sm_scale * kLog2e;
                    unsigned char* q = smem + C::kOffQ;
                    const int rl = C::kNQ + row;
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
        };

        dead |= !wait(&sm.seg_full[0], 0);
        if (!all_any<C::kSoft>(dead)) {
            convert(0, sm.segs[0]);
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
                float2 qs[kRW / 2];  // (read from shared memory for each tile: R = 16 1%, 32 2% longer)
#pragma unroll
                for (int r = 0; r < kRW; r += 2)
                    qs[r / 2] = *reinterpret_cast<const float2*>(&sm.qs[k & 1][r0 + r]);
                bool first = true;
                for (int t = seg.tile0; t < tile1; ++t, ++g, first = false) {
                    const int b = g & 1, me = g % kMetas;
                    dead |= !wait(&sm.meta_full[me], (uint32_t)(g / kMetas) & 1);
                    const float4 sc = sm.meta[me][page_at];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.meta_empty[me]);
                    const int pos = t * kTileKeys + key;
                    const bool in = pos < keys;
                    const float ks = in ? sc.x : 0.f;
                    const float lvs = in ? sc.y : 0.f, inv = in ? sc.z : 0.f;
                    const bool cut = (t + 1) * kTileKeys > lim_min;  // some row does not see all
                    dead |= !wait(&sm.s_full[b], (uint32_t)(g >> 1) & 1);
                    tc_fence_after();
                    // scores in base 2 with the value scale, less their row's reference
                    float x[kRW];
                    {
                        const float2 kk = make_float2(ks, ks), lv = make_float2(lvs, lvs);
                        constexpr int kN = kRW < 16 ? kRW : 16;
#pragma unroll
                        for (int q = 0; q < kRW; q += kN) {
                            float u[1][kN];
                            tmem_ld_start<kN>(lanes + b * C::kNQ + r0 + q, u[0]);
                            tmem_ld_wait<kN, 1>(u);
#pragma unroll
                            for (int i = 0; i < kN; i += 2) {
                                const float2 m = *reinterpret_cast<const float2*>(sm.mref + r0 + q + i);
                                const float2 z = mul_f32x2(make_float2(u[0][i], u[0][i + 1]), qs[(q + i) / 2]);
                                const float2 y = fma_f32x2(z, kk, add_f32x2(lv, m));
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
                    const int half = C::kPHalves ? b * 64 : 0;
                    unsigned char* pt = smem + C::kOffP + (C::kPHalves ? 0 : b * C::kPBytes) + key * 128;
                    auto p_chunk = [&](int byte) {  // 16 bytes of the row
                        return reinterpret_cast<uint4*>(pt + ((((half + byte) >> 4) ^ (key & 7)) << 4));
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
                            const __half2 up5 = __float2half2_rn(32.f);
                            const __half2 d1 = __hmul2(__hsub2(p, as_half2(e4m3_to_half2(e0))), up5);
                            const uint16_t e1 = half2_to_e4m3(as_u32(d1));
                            const __half2 d2 = __hsub2(d1, as_half2(e4m3_to_half2(e1)));
                            const uint16_t e2 = half2_to_e4m3(as_u32(__hfma2(d2, up5, place)));
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
                if (more) convert(kn, sm.segs[kn % kSegs]);
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
                    // (where no tile was read, the warps that convert values may not have reset it yet)
                    const int nan_from = some ? sm.first_nan[k % kSegs][key] : INT32_MAX;
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
                                if constexpr (C::kTerms == 3) y += o[1][i] * 0x1p-5f + o[2][i] * 0x1p-10f;
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

// Rows of a tile: the least that holds a key head's rows of the longest run.  Up to 32 rows are
// columns of the tiles (this file's kernel), more are lanes (the wide kernel, one row a thread).
// Four rows a head (64 decode requests, 615 MB of cache): R = 8 takes 111.5 us, 16 114, 32 165, 64
// 198, 128 235, 256 315.  Up to 64 rows (128 requests, 565 MB): R = 64 takes 150 us, 128 174, 256 247,
// and several tiles a unit 200 (32) and 220 (16); 64 rows as columns of f16 tiles took 184.
// The whole call takes the longest run's tile.  That is right where runs are about equal; in a mixed
// batch the short runs pay for it: 62 decode requests take 121 us and two chunks of 1,000 tokens 241
// in calls of their own, 505 in one; 112 single tokens 99 and 16 runs of 8 tokens 39, 163 in one.
int tile_rows(int heads, int kv_heads, int max_run) {
    const int64_t rows = (int64_t)(heads / kv_heads) * std::max(max_run, 1);
    return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256;
}
template <int R>
constexpr int ctas_of() { return kPlanSMs * Cfg<R>::kCtasPerSm; }

template <int R>
cudaError_t launch_rows(const AttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, bool join,
                        int* status, cudaStream_t stream) {
    static std::atomic<uint64_t> raised{0};
    cudaError_t e = raise_smem(paged_attention_kernel<R>, smem_bytes<R>(), raised);
    if (e != cudaSuccess) return e;
    paged_attention_kernel<R><<<ctas_of<R>(), Cfg<R>::kThreads, smem_bytes<R>(), stream>>>(a, km, vm, status);
    e = cudaGetLastError();
    return e == cudaSuccess && join ? launch_join<R>(a, ctas_of<R>(), stream) : e;
}

}  // namespace

size_t paged_attention_workspace(int32_t heads, int32_t kv_heads, int32_t max_run) {
    switch (tile_rows(heads, kv_heads, max_run)) {
        case 8: return workspace_of<8>(ctas_of<8>());
        case 16: return workspace_of<16>(ctas_of<16>());
        case 32: return workspace_of<32>(ctas_of<32>());
        default: return paged_attention_wide_workspace(tile_rows(heads, kv_heads, max_run));
    }
}

cudaError_t launch_paged_attention(const AttnArgs& a, int* status, cudaStream_t stream,
                                   uint64_t* launches) {
    CUtensorMap km, vm;
    if (!make_map(&km, a.k_cache, a) || !make_map(&vm, a.v_cache, a)) return cudaErrorInvalidValue;
    // units of up to kSnapUnit tiles are never cut: where the table holds no longer ones, nothing
    // is left to join
    const bool join = (int64_t)a.width * a.page_size > kSnapUnit * kTileKeys;
    *launches += join ? 2 : 1;
    const int rows = tile_rows(a.heads, a.kv_heads, a.max_run);
    switch (rows) {
        case 8: return launch_rows<8>(a, km, vm, join, status, stream);
        case 16: return launch_rows<16>(a, km, vm, join, status, stream);
        case 32: return launch_rows<32>(a, km, vm, join, status, stream);
        default: return launch_paged_attention_wide(rows, a, km, vm, join, status, stream);
    }
}

}  // namespace kda
