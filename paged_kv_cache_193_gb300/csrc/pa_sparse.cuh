// Shared by the block-sparse decode sources: limits, and host-side launch
// helpers.
#pragma once

#include <atomic>

#include "pa_launch.cuh"

namespace pa {
namespace sparse {

// Exponents of the int8 bounds.  With both sides in this range and the whole
// number below 2^22, a score is exact in fp32 and never out of its range.
constexpr int kMinExp = -60, kMaxExp = 40;
// Marks a page whose keys hold an infinity or NaN: its score is +infinity.
constexpr int kOddExp = 127;

constexpr int kSms = 152;

// Longest block-table row of the choice: a cluster of eight CTAs keeps one
// 32-bit key per page, 64 KB to a CTA beside its copies in flight.
constexpr int kMaxKeys = 16384;
constexpr int kMaxTableBlocks = 8 * kMaxKeys;

// ---- thread-block clusters and distributed shared memory ----------------------

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// fp32 at shared-memory address `addr` of the cluster's CTA `rank`
__device__ __forceinline__ float ld_cluster(uint32_t addr, uint32_t rank) {
    float x;
    asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %1, %2;\n\t"
                 "ld.shared::cluster.f32 %0, [r];\n\t}"
                 : "=f"(x)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return x;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr, uint32_t rank) {
    return __float_as_uint(ld_cluster(addr, rank));
}
__device__ __forceinline__ uint4 ld_cluster_v4(uint32_t addr, uint32_t rank) {
    uint4 v;
    asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %4, %5;\n\t"
                 "ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [r];\n\t}"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t rank, uint32_t x) {
    asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, %1;\n\t"
                 "st.shared::cluster.u32 [r], %2;\n\t}" ::"r"(addr), "r"(rank), "r"(x)
                 : "memory");
}
__device__ __forceinline__ uint32_t atom_add_cluster(uint32_t addr, uint32_t rank, uint32_t x) {
    uint32_t old;
    asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %1, %2;\n\t"
                 "atom.relaxed.cluster.shared::cluster.add.u32 %0, [r], %3;\n\t}"
                 : "=r"(old)
                 : "r"(addr), "r"(rank), "r"(x)
                 : "memory");
    return old;
}

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
}  // namespace sparse
}  // namespace pa
