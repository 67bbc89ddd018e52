// Shared by the block-sparse decode sources: limits, and host-side launch
// helpers.
#pragma once

#include <atomic>

#include "pa_device.cuh"

namespace pa {
namespace sparse {

// Exponents of the int8 bounds.  With both sides in this range and the whole
// number below 2^22, a score is exact in fp32 and never out of its range.
constexpr int kMinExp = -60, kMaxExp = 40;
// Marks a page whose keys hold an infinity or NaN: its score is +infinity.
constexpr int kOddExp = 127;

// Longest block-table row of the choice: a cluster of eight CTAs keeps one
// 32-bit key per page, 128 KB to a CTA.
constexpr int kMaxTableBlocks = 8 * 32768;
constexpr int kMaxSelectSmem = 32768 * 4;

// Raise a kernel's dynamic shared-memory limit once per device; `done` is a
// flag word of the kernel's own (the first call on a device should precede
// any stream capture).
inline pa_status raise_smem_limit(const void *kernel, int bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    pa_status st = cuda_check(cudaGetDevice(&dev), "cudaGetDevice");
    if (st != PA_OK) return st;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0;
    if (bit && (done.load(std::memory_order_acquire) & bit)) return PA_OK;
    st = cuda_check(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes),
                    "cudaFuncSetAttribute");
    if (st == PA_OK) done.fetch_or(bit, std::memory_order_release);
    return st;
}

pa_status check_select(int num_rows, int num_q_heads, int num_kv_heads, int head_dim, int num_blocks,
                       int block_size, int max_blocks, int top_k, int sink, int recent);
pa_status run_select(const void *q, const int8_t *summary, const int8_t *exponents,
                     const int32_t *block_tables, int max_blocks, const int32_t *context_lens,
                     int num_rows, int num_q_heads, int num_kv_heads, int head_dim, int num_blocks,
                     int block_size, int top_k, int sink, int recent, int32_t *selected,
                     int32_t *counts, cudaStream_t stream);

}  // namespace sparse
}  // namespace pa
