// kda_paged.cuh — launchers of the paged serving operators (page plan, 8-bit cache append, paged
// attention, draft verification), called by kda_api.cu, and what their kernels share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/kda.h"

namespace kda {

constexpr int kPlanMaxSeqs = 8192;  // requests of one page plan (24 bytes of shared memory each)

// Page sizes the kernels take: a tile of 128 keys is a whole number of pages, and a page a whole
// number of the 8-row groups of a swizzled tile.
inline bool page_size_ok(int32_t bs) { return bs == 16 || bs == 32 || bs == 64 || bs == 128; }

struct PlanArgs {
    int32_t num_seqs, width, page_size, capacity;
    int64_t total_tokens;
    const int32_t *cached, *cu, *release, *held;
    int32_t *tables, *free_list;
    const int32_t* free_count;
    int32_t *context, *held_out, *free_out, *positions, *slots;
};
cudaError_t launch_paged_plan(const PlanArgs& a, int* status, cudaStream_t stream);

struct AppendArgs {
    int64_t total_tokens;
    int32_t kv_heads, page_size, num_pages;
    const void *k, *v;          // bf16 [T][kv_heads][128], tokens k_stride / v_stride elements apart
    int64_t k_stride, v_stride;
    const int32_t* slots;
    uint8_t *k_cache, *v_cache;  // e4m3 [num_pages][kv_heads][page_size][128]
    float *k_scale, *v_scale;    // [num_pages][kv_heads]
};
cudaError_t launch_paged_append(const AppendArgs& a, int* status, cudaStream_t stream);

// Keys of a table row and rows of a call: whole tiles of 128 keys and 256 rows stay within 31 bits.
constexpr int32_t kMaxAttnKeys = INT32_MAX - 127, kMaxAttnRows = INT32_MAX - 255;

struct AttnArgs {
    int32_t num_seqs, heads, kv_heads, page_size, num_pages, width, max_run;
    int64_t total_tokens;
    float sm_scale;
    const void* q;              // bf16 [T][heads][128], tokens q_stride elements apart
    int64_t q_stride;
    const int32_t *cu, *tables, *context;
    const uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    void* out;                  // bf16 [T][heads][128]
    void* workspace;
};
size_t paged_attention_workspace(int32_t heads, int32_t kv_heads, int32_t max_run);
cudaError_t launch_paged_attention(const AttnArgs& a, int* status, cudaStream_t stream,
                                   uint64_t* launches);

constexpr int32_t kMaxVocab = 1 << 30;  // a thread's stride past the last entry stays within 31 bits

struct VerifyArgs {
    int32_t num_seqs, vocab, dtype;
    int64_t total_tokens;
    const void *p, *q;          // [T][vocab]; q may be null (certain drafts)
    const int32_t *tokens, *cu;
    const float *uniform, *noise;
    int32_t *commit, *next, *out;
};
cudaError_t launch_verify_draft(const VerifyArgs& a, int* status, cudaStream_t stream);

// The shared memory that launches of a kernel may ask for, raised once per device to the most that any
// of them asks: the attribute is the kernel's, not a launch's, and shared by all host threads.
template <class Kernel>
cudaError_t raise_smem(Kernel kernel, size_t bytes, std::atomic<uint64_t>& raised) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (raised.load() & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) raised.fetch_or(bit);
    return e;
}

// The request that packed row t belongs to: the last n with cu[n] <= t (empty runs before it have
// cu[n] == cu[n + 1]).  t < cu[num_seqs].
__device__ __forceinline__ int seq_of_row(const int32_t* cu, int num_seqs, int t) {
    int lo = 0, hi = num_seqs;  // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}

}  // namespace kda
