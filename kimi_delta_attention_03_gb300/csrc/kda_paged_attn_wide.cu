// kda_paged_attn_wide.cu — paged attention for more than 32 rows of a key head: long drafts of many
// query heads, chunks of a prompt.  The mathematics, the shares of work and the partial results
// are those of kda_paged_attn.cu; here the rows are the lanes of the tiles.
//
//   S [128 rows x 128 keys] = [Q_hi | Q_lo] [K | K]^T    K's tile as TMA wrote it; Q_hi e4m3, Q_lo
//                                                        e5m2, which reaches 2^7 times lower and so
//                                                        holds what Q_hi leaves of a bf16 q
//   O [128 rows x 128 channels] += P V                   f16: P from tensor memory, where it takes
//                                                        the place of S, V widened once per tile
//
// A thread has one row, so maxima and sums never leave it: no barrier and no vote beyond its warp.
// A warp raises its rows' references (and rescales their lanes of O) only where a score exceeds one
// by 2^11.5; f16 has the room for that.
//
// Two chains of S and O share the tensor cores, so that one multiplies while the other's warps take
// exponentials:
//   R = 64   both chains have the unit's rows, chain 0 its even tiles on lanes 0-63, chain 1 its odd
//            tiles on lanes 64-127 (each on two warps, all four schedulers busy); joined at the end
//   R = 128  the same with all lanes and four warps each
//   R = 256  chain 0 has rows 0-127, chain 1 rows 128-255, both every tile
// Four more warps widen the values and, a segment ahead, split the rows of q into their terms.
//
// What bounds it: shared memory and the chain's own order, before HBM.  Per tile of 128 keys the
// tensor cores want 512 cycles for the scores and 512 for the weighted sums of 128 lanes; shared
// memory carries both terms of Q against K (64 KB), V (32 KB), its widening (48 KB) and what TMA
// writes (32 KB), 1408 cycles of 128 bytes.  A chain's softmax takes about 2100 cycles and its two
// products 1400 to 1800, one after the other as P takes S's place, and two chains overlap.
//     R = 64   128 requests of up to 64 rows a head, 565 MB of cache: 150 us, 3.8 TB/s, 56% of the
//              measured copy bandwidth (a tile every 1950 cycles; HBM alone would allow 1400)
//     R = 256  three chunks of about 1000 tokens over 6000 to 8000: 338 us, 1000 TFLOP/s (of
//              1937 measured for bf16), of which the joining of cut units takes 11
// Measured and not kept: two threads a row (152 us and 388), scores 64 keys at a time with Q in
// tensor memory (236 and 482), two 64-key buffers of scores a chain (278 and 520), scores loaded a
// chunk ahead (160 and 356), an issuer for each chain (170 and 446),
// the weighted sum of a tile's first half issued before its second half's weights (165 and 338).
#include <algorithm>
#include <atomic>

#include "kda_paged_attn.cuh"

namespace kda {
namespace {

using namespace attn;

// Weights are 2^kPeak at their row's reference and may reach 2^(kPeak + kSlack) < 65504.
constexpr float kPeak = 4.f, kSlack = 11.5f;
constexpr int kStageLd = 17;  // floats between rows of a chain's staging buffer

template <int R>
struct Wide {
    static constexpr bool kPair = R == 256;                 // a chain has its own rows
    static constexpr int kChain = R == 64 ? 64 : 128;       // threads of a chain, one row each
    static constexpr int kSoft = 2 * kChain;                // softmax threads
    static constexpr int kConv = 128;                       // threads that convert values and q
    static constexpr int kThreads = kSoft + kConv + 64;     // and the producer's and the issuer's
    static constexpr int kKStages = R == 128 ? 2 : 3, kVStages = 2;
    static constexpr int kQBufs = kPair ? 1 : 2;            // segments whose q is held
    static constexpr int kQBytes = (kPair ? 2 : 1) * 2 * kTileBytes;  // per 128 lanes: hi, lo
    static constexpr uint32_t kOffK = 0;
    static constexpr uint32_t kOffV = kOffK + kKStages * kTileBytes;
    static constexpr uint32_t kOffVal = kOffV + kVStages * kTileBytes;
    static constexpr uint32_t kOffQ = kOffVal + 2 * 2 * kTileBytes;
    static constexpr uint32_t kOffStage = kOffQ + kQBufs * kQBytes;
    static constexpr uint32_t kOffSmall = kOffStage + (kPair ? 0 : 2 * R * kStageLd * 4);
};

template <int R>
struct WideSmall : Ring<Wide<R>::kKStages, Wide<R>::kVStages, Wide<R>::kThreads> {
    uint64_t s_full[2], p_ready[2], pv_done[2], val_empty[2];
    uint64_t q_full[Wide<R>::kQBufs], q_empty[Wide<R>::kQBufs], qs_full[kSegs];
    float qs[kSegs][R];                          // score scale of each row: sm_scale log2 e / s
    float m[Wide<R>::kSoft], l[Wide<R>::kSoft];  // what the other chain's thread has
};
template <int R>
constexpr size_t wide_smem() { return Wide<R>::kOffSmall + sizeof(WideSmall<R>) + 1024; }
static_assert(wide_smem<64>() <= 232448 && wide_smem<128>() <= 232448 && wide_smem<256>() <= 232448, "shared memory of a CTA");

__device__ __forceinline__ void ld32_start(uint32_t addr, float (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
          "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
          "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]),
          "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]),
          "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(addr) : "memory");
}
__device__ __forceinline__ void ld32_wait(float (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(r[i]));
}

template <int R>
__global__ void __launch_bounds__(Wide<R>::kThreads, 1)
paged_attention_wide_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap k_map,
                            const __grid_constant__ CUtensorMap v_map, int* status) {
    using C = Wide<R>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    WideSmall<R>& sm = *reinterpret_cast<WideSmall<R>*>(smem + C::kOffSmall);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kProducer = (C::kSoft + C::kConv) / 32, kIssuer = kProducer + 1;
    const int group = a.heads / a.kv_heads, shift = 31 - __clz(a.page_size);
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
        sm.init(C::kConv / 32, (C::kPair ? C::kSoft : C::kChain) / 32, (C::kSoft + C::kConv) / 32 + 1,
                C::kConv, 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm.s_full[b], 1);
            mbar_init(&sm.p_ready[b], C::kChain);
            mbar_init(&sm.pv_done[b], 1);
            mbar_init(&sm.val_empty[b], 1);
        }
        for (int b = 0; b < C::kQBufs; ++b) {
            mbar_init(&sm.q_full[b], C::kConv);
            mbar_init(&sm.q_empty[b], 1);
        }
        for (int b = 0; b < kSegs; ++b) mbar_init(&sm.qs_full[b], C::kConv);
        mbar_init_fence();
        tma_prefetch_desc(&k_map);
        tma_prefetch_desc(&v_map);
    }
    if (warp == kIssuer) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    fence_async_shared();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;  // columns: S / P of chains 0 and 1, then O of chains 0 and 1
    const Waiter wait = {&sm.abort_flag, status};

    if (warp == kProducer) {
        produce<R, C::kKStages, C::kVStages, false>(a, sm, smem, C::kOffK, C::kOffV, 0, k_map, v_map,
                                                    descs, wait, status);
    } else if (warp == kIssuer) {
        // ------------------------------------------------------------------------ MMA issuer
        // The whole warp walks the work with values that are the same in every lane, so that the
        // descriptors are formed in uniform registers, and one elected lane issues: a thread on its
        // own needs more than the 64 cycles that a multiplication takes to issue the next.
        {
            constexpr uint32_t kIdHi = idesc_zero(kTileKeys, false, false);
            constexpr uint32_t kIdLo = kIdHi | 1u << 7;  // the first operand in e5m2
            constexpr uint32_t kIdO = idesc_zero(kDim, false, true);
            const uint32_t base = __shfl_sync(~0u, saddr(smem), 0), tm = __shfl_sync(~0u, tmem, 0);
            int done[2] = {0, 0};   // tiles of each chain
            int open[2] = {-1, -1}; // tile whose weights are awaited,
            bool fresh[2] = {};     // and whether it is the chain's first of its segment
            int chains = 2;         // chains with rows
            uint32_t q_at = 0;      // this segment's q
            auto sums = [&](int ch, bool ok) {  // ok: how the waits before it ended
                const int g = open[ch], b = g & 1;
                // (both asked before either answer is looked at)
                const bool v = mbar_try_wait(&sm.val_full[b], (uint32_t)(g >> 1) & 1);
                const bool p = mbar_try_wait(&sm.p_ready[ch], (uint32_t)(done[ch] - 1) & 1);
                ok &= v || wait.slow(&sm.val_full[b], (uint32_t)(g >> 1) & 1);
                ok &= p || wait.slow(&sm.p_ready[ch], (uint32_t)(done[ch] - 1) & 1);
                if (!__all_sync(~0u, ok)) return false;  // the lanes leave together
                tc_fence_after();
                const uint64_t v_desc = smem_desc(base + C::kOffVal + b * 2 * kTileBytes, 16384, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)  // 16 keys each: 8 columns of P, 16 rows of V
                        mma_ts(tm + 256 + ch * 128, tm + ch * 128 + 8 * i, v_desc + 128 * i, kIdO,
                               !fresh[ch] || i > 0);
                    if (!C::kPair || ch == chains - 1) mma_commit(&sm.val_empty[b]);
                    mma_commit(&sm.pv_done[ch]);
                }
                __syncwarp();
                open[ch] = -1;
                return true;
            };
            // Scores of a tile.  P takes the place of S, so the chain's last weighted sum goes first.
            auto scores = [&](int ch, int g, bool first) {
                const int s = g % C::kKStages;
                // (chain 1 of R = 256 follows chain 0 on the same keys)
                const bool ok = (C::kPair && ch == 1) || wait(&sm.k_full[s], (uint32_t)(g / C::kKStages) & 1);
                if (open[ch] >= 0) {
                    if (!sums(ch, ok)) return false;
                } else {
                    if (!__all_sync(~0u, ok)) return false;
                    tc_fence_after();
                }
                const uint64_t k_desc = smem_desc(base + C::kOffK + s * kTileBytes, 16, 1024);
                const uint64_t q_desc = smem_desc(base + q_at + (C::kPair ? ch * 2 * kTileBytes : 0), 16, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)  // 32 channels each: the four of Q_hi, the four of Q_lo
                        mma_f8(tm + ch * 128, q_desc + (i >> 2) * (kTileBytes >> 4) + 2 * (i & 3),
                               k_desc + 2 * (i & 3), i < 4 ? kIdHi : kIdLo, i > 0);
                    if (!C::kPair || ch == chains - 1) mma_commit(&sm.k_empty[s]);
                    mma_commit(&sm.s_full[ch]);
                }
                __syncwarp();
                open[ch] = g;
                fresh[ch] = first;
                ++done[ch];
                return true;
            };
            int g = 0;
            for (int k = 0;; ++k) {
                if (!wait.warp(&sm.seg_full[k % kSegs], (uint32_t)(k / kSegs) & 1)) break;
                const Seg& seg = sm.segs[k % kSegs];
                const int n = __shfl_sync(~0u, seg.n, 0), tiles = __shfl_sync(~0u, seg.tile1 - seg.tile0, 0);
                const int rows = __shfl_sync(~0u, seg.rows, 0);
                // The last segment's weighted sums go first: its outputs, which the softmax warps
                // are at now, come before their next scores.
                bool ok = true;
                const int early = !C::kPair && open[0] > open[1] ? 1 : 0;
                for (int i = 0; i < 2 && ok; ++i)
                    if (open[early ^ i] >= 0) ok = sums(early ^ i, true);
                if (!ok || n < 0) break;
                if (lane == 0) mbar_arrive(&sm.seg_empty[k % kSegs]);
                __syncwarp();
                chains = C::kPair && rows <= 128 ? 1 : 2;
                const int qb = k % C::kQBufs;
                q_at = C::kOffQ + qb * C::kQBytes;
                if (!wait.warp(&sm.q_full[qb], (uint32_t)(k / C::kQBufs) & 1)) break;
                tc_fence_after();
                const int g0 = g;
                for (; g < g0 + tiles && ok; ++g) {
                    if constexpr (C::kPair)
                        for (int ch = 0; ch < chains && ok; ++ch) ok = scores(ch, g, g == g0);
                    else
                        ok = scores(g & 1, g, g < g0 + 2);
                }
                if (!ok) break;
                if (elect_one()) mma_commit(&sm.q_empty[qb]);  // (at once where the segment has no tile)
                __syncwarp();
            }
        }
        __syncwarp();
    } else if (warp >= C::kSoft / 32) {
        // --------------------------------------------------------------- values and rows of q
        // Rows of q as an e4m3 and an e5m2 term, each row scaled by a power of two s so that its
        // largest lies in [128, 256): eight threads a row, 16 channels each.
        const int thread = tid - C::kSoft;
        auto split_q = [&](int k, const Seg& sg) {
            const int qb = k % C::kQBufs;
            if (k >= C::kQBufs && !wait(&sm.q_empty[qb], (uint32_t)(k / C::kQBufs - 1) & 1)) return false;
            const int j = thread & 7;
            constexpr int kStep = C::kConv / 8;  // rows at a time; the loads of four steps go together
#pragma unroll 1
            for (int row0 = thread >> 3; row0 < R; row0 += 4 * kStep) {
                uint4 all[4][2];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = row0 + i * kStep, r = sg.row0 + row;
                    all[i][0] = all[i][1] = make_uint4(0, 0, 0, 0);
                    if (row < sg.rows) {
                        const uint4* p = reinterpret_cast<const uint4*>(
                            static_cast<const __nv_bfloat16*>(a.q) + (int64_t)(sg.q0 + r / group) * a.q_stride +
                            (sg.head * group + r % group) * kDim + j * 16);
                        all[i][0] = __ldg(p);
                        all[i][1] = __ldg(p + 1);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = row0 + i * kStep;
                    const uint4 (&x)[2] = all[i];
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
                    // 128 lanes a tile; R = 64 has its rows in both halves
                    unsigned char* q = smem + C::kOffQ + qb * C::kQBytes + (row >> 7) * 2 * kTileBytes;
#pragma unroll
                    for (int at = row & 127; at < 128; at += R == 64 ? 64 : 128) {
                        unsigned char* to = q + at * 128 + ((j ^ (at & 7)) << 4);
                        *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(to + kTileBytes) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                    if (j == 0)
                        sm.qs[k % kSegs][row] = __int_as_float((127 - 134 + e) << 23) * a.sm_scale * kLog2e;
                }
            }
            fence_async_shared();
            mbar_arrive(&sm.q_full[qb]);
            // (on a ring of its own: q_full can be two segments ahead of the softmax warps)
            mbar_arrive(&sm.qs_full[k % kSegs]);
            return true;
        };
        convert_values<C::kVStages>(sm, smem, C::kOffV, C::kOffVal, sm.val_empty, thread, group, wait, split_q);
    } else {
        // --------------------------------------------------------- scores, weights and outputs
        const int ch = tid / C::kChain;                             // chain
        const int row = C::kPair ? tid : tid & (R - 1);             // row of the unit
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // lane tid % 128 of the tiles
        const uint32_t s_col = lanes + ch * 128, o_col = lanes + 256 + ch * 128;
        bool dead = false;  // a wait gave up: run on to where all warps can leave together
        int g = 0, done = 0;  // tiles so far; of this chain
        {
            for (int k = 0;; ++k) {
                dead |= !wait(&sm.seg_full[k % kSegs], (uint32_t)(k / kSegs) & 1);
                if (all_any<C::kSoft>(dead)) break;
                const Seg& seg = sm.segs[k % kSegs];
                if (seg.n < 0) break;
                dead |= !wait(&sm.qs_full[k % kSegs], (uint32_t)(k / kSegs) & 1);
                const float qs = sm.qs[k % kSegs][row];
                const int lim_min = seg.lim0 + seg.row0 / group, tile1 = seg.tile1;
                const int lim = row < seg.rows ? seg.lim0 + (seg.row0 + row) / group : 0;
                const bool active = !C::kPair || ch * 128 < seg.rows;
                float m = 0.f, l = 0.f;
                int mine = 0;  // tiles of this chain in the segment
                for (int t = seg.tile0; t < tile1; ++t, ++g) {
                    if (!C::kPair && (g & 1) != ch) continue;
                    const int me = g % kMetas;
                    dead |= !wait(&sm.meta_full[me], (uint32_t)(g / kMetas) & 1);
                    if (active) {
                        const bool cut = (t + 1) * kTileKeys > lim_min;  // some row does not see all
                        // scales of a chunk's pages, read a chunk ahead: shared memory is busy with
                        // operands, and a load from it takes up to 300 cycles
                        float4 page[2], next[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) next[h] = sm.meta[me][(h * 16) >> shift];
                        dead |= !wait(&sm.s_full[ch], (uint32_t)done & 1);
                        tc_fence_after();
                        // rolled: four copies of the body do not stay in the instruction cache
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            float x[32];
                            ld32_start(s_col + c * 32, x);
                            ld32_wait(x);
                            // scores in base 2 with the value scale, less the row's reference
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                page[h] = next[h];
                                const float2 cc = make_float2(page[h].x * qs, page[h].x * qs);
                                const float2 bb = make_float2(page[h].y - m, page[h].y - m);
#pragma unroll
                                for (int i = h * 16; i < h * 16 + 16; i += 2) {
                                    const float2 y = fma_f32x2(make_float2(x[i], x[i + 1]), cc, bb);
                                    x[i] = y.x;
                                    x[i + 1] = y.y;
                                }
                            }
#pragma unroll
                            for (int h = 0; h < 2; ++h) next[h] = sm.meta[me][(min(c + 1, 3) * 32 + h * 16) >> shift];
                            if (cut) {
                                const int rel = lim - t * kTileKeys - c * 32;
#pragma unroll
                                for (int i = 0; i < 32; ++i) x[i] = i < rel ? x[i] : -INFINITY;
                            }
                            float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                            for (int i = 4; i < 32; i += 2)
                                asm("max.f32 %0, %0, %1, %2;" : "+f"(top[(i >> 1) & 3]) : "f"(x[i]), "f"(x[i + 1]));
                            top[0] = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                            const bool first = c == 0 && mine == 0;
                            if (__builtin_expect(__any_sync(~0u, top[0] > kPeak + kSlack || first), 0)) {
                                // the reference rises by what the largest score is above 2^kPeak; the
                                // segment's first 32 keys set it.  A row that sees none of those sees
                                // none in the segment.
                                float up = first ? top[0] - kPeak : fmaxf(top[0] - kPeak, 0.f);
                                if (!(up > -1e37f)) up = first ? kNoRef : 0.f;
                                m += up;
#pragma unroll
                                for (int i = 0; i < 32; ++i) x[i] -= up;
                                if (!first) {
                                    const float f = ex2_approx(-up);
                                    l *= f;
                                    if (c > 0) {  // this tile's weights so far
                                        tmem_st_wait();
#pragma unroll 1
                                        for (int j = 0; j < c * 16; j += 8) {
                                            float p[1][8];
                                            tmem_ld_start<8>(s_col + j, p[0]);
                                            tmem_ld_wait<8, 1>(p);
#pragma unroll
                                            for (int i = 0; i < 8; ++i) {
                                                const float2 y = __half22float2(as_half2(__float_as_uint(p[0][i])));
                                                p[0][i] = __uint_as_float(as_u32(__floats2half2_rn(y.x * f, y.y * f)));
                                            }
                                            tmem_st8(s_col + j, p[0]);
                                        }
                                    }
                                    if (mine > 0) {
                                        dead |= !wait(&sm.pv_done[ch], (uint32_t)(done - 1) & 1);
                                        tc_fence_after();
#pragma unroll 1
                                        for (int j = 0; j < kDim; j += 16) {
                                            float o[1][16];
                                            tmem_ld_start<16>(o_col + j, o[0]);
                                            tmem_ld_wait<16, 1>(o);
                                            uint32_t y[16];
#pragma unroll
                                            for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(o[0][i] * f);
                                            tmem_st16(o_col + j, y);
                                        }
                                    }
                                    tmem_st_wait();
                                }
                            }
                            // weights as f16 and their sums
                            uint32_t p[16];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                                for (int i = h * 16; i < h * 16 + 16; i += 2) {
                                    const float2 y = make_float2(ex2_approx(x[i]), ex2_approx(x[i + 1]));
                                    sum = add_f32x2(sum, y);
                                    p[i >> 1] = as_u32(__floats2half2_rn(y.x, y.y));
                                }
                                l = fmaf(sum.x + sum.y, page[h].z, l);
                            }
                            tmem_st16(s_col + c * 16, p);
                        }
                        tmem_st_wait();
                        tc_fence_before();
                        mbar_arrive(&sm.p_ready[ch]);
                        ++done;
                        ++mine;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.meta_empty[me]);
                }
                // outputs: this thread's row, 32 channels at a time
                if (mine > 0) {
                    dead |= !wait(&sm.pv_done[ch], (uint32_t)(done - 1) & 1);
                    tc_fence_after();
                } else {
                    m = kNoRef;
                }
                float f = 1.f;
                if (!C::kPair) {
                    sm.m[tid] = m;
                    sm.l[tid] = l;
                    all_any<C::kSoft>(false);  // both chains' last sums, and so all values, are done
                }
                const bool nans = all_any<C::kSoft>(sm.first_nan[k % kSegs][tid & 127] != INT32_MAX);
                if (!C::kPair) {
                    const float other = sm.m[tid ^ R], both = fmaxf(m, other);
                    f = ex2_approx(m - both);
                    l = f * l + ex2_approx(other - both) * sm.l[tid ^ R];
                    m = both;
                }
                const bool writes = row < seg.rows;
                const float scale = seg.slot >= 0 ? 1.f : l == 0.f ? 0.f : 1.f / l;
                const int r = seg.row0 + row;
                const int64_t to = (int64_t)(seg.q0 + r / group) * a.heads + seg.head * group + r % group;
                // 16 channels at a time.  Where both chains have the row, each gives out half of its
                // channels: what the other has of them comes through shared memory.
                float* stage = reinterpret_cast<float*>(smem + C::kOffStage) + row * kStageLd;
                constexpr int kChannels = C::kPair ? kDim : kDim / 2;
#pragma unroll 1
                for (int j = 0; j < kChannels; j += 16) {
                    const int c = C::kPair ? j : ch * kChannels + j;
                    float o[C::kPair ? 1 : 2][16];
                    if (mine > 0) {
                        tmem_ld_start<16>(o_col + c, o[0]);
                        if constexpr (!C::kPair) tmem_ld_start<16>(o_col + (c ^ kChannels), o[1]);
                        tmem_ld_wait(o);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[0][i] = mine > 0 ? o[0][i] * f : 0.f;
                    if constexpr (!C::kPair) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) stage[ch * R * kStageLd + i] = mine > 0 ? o[1][i] * f : 0.f;
                        all_any<C::kSoft>(false);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[0][i] += stage[(ch ^ 1) * R * kStageLd + i];
                        all_any<C::kSoft>(false);
                    }
                    if (!writes) continue;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        o[0][i] *= scale;
                        if (nans && lim > sm.first_nan[k % kSegs][c + i]) o[0][i] = NAN;
                    }
                    if (seg.slot >= 0) {
                        float4* p = reinterpret_cast<float4*>(&parts[seg.slot].o[row][c]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            p[i] = make_float4(o[0][4 * i], o[0][4 * i + 1], o[0][4 * i + 2], o[0][4 * i + 3]);
                    } else {
                        uint4* p = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + to * kDim + c);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            p[i] = make_uint4(
                                pack_bf16(o[0][8 * i], o[0][8 * i + 1]), pack_bf16(o[0][8 * i + 2], o[0][8 * i + 3]),
                                pack_bf16(o[0][8 * i + 4], o[0][8 * i + 5]), pack_bf16(o[0][8 * i + 6], o[0][8 * i + 7]));
                    }
                }
                if (writes && (C::kPair || ch == 0) && seg.slot >= 0) {
                    parts[seg.slot].m[row] = m;
                    parts[seg.slot].l[row] = l;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.seg_empty[k % kSegs]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kIssuer) tmem_dealloc(tmem, 512);
}

template <int R>
cudaError_t launch_wide(const AttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, bool join,
                        int* status, cudaStream_t stream) {
    static std::atomic<uint64_t> raised{0};
    cudaError_t e = raise_smem(paged_attention_wide_kernel<R>, wide_smem<R>(), raised);
    if (e != cudaSuccess) return e;
    paged_attention_wide_kernel<R><<<kPlanSMs, Wide<R>::kThreads, wide_smem<R>(), stream>>>(a, km, vm, status);
    e = cudaGetLastError();
    return e == cudaSuccess && join ? launch_join<R>(a, kPlanSMs, stream) : e;
}

}  // namespace

size_t paged_attention_wide_workspace(int rows) {
    return rows == 64 ? workspace_of<64>(kPlanSMs)
           : rows == 128 ? workspace_of<128>(kPlanSMs) : workspace_of<256>(kPlanSMs);
}

cudaError_t launch_paged_attention_wide(int rows, const AttnArgs& a, const CUtensorMap& k_map,
                                        const CUtensorMap& v_map, bool join, int* status,
                                        cudaStream_t stream) {
    return rows == 64 ? launch_wide<64>(a, k_map, v_map, join, status, stream)
           : rows == 128 ? launch_wide<128>(a, k_map, v_map, join, status, stream)
                         : launch_wide<256>(a, k_map, v_map, join, status, stream);
}

}  // namespace kda
