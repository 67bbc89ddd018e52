// Cross attention: every row of a sequence attends to all of an encoder's
// states, whose keys and values lie in the paged cache ("vLLM PagedAttention:
// Memory Optimization & High-Throughput LLM Inference Tuning", section 2: the
// cache is read through the sequence's block table).
//
// The rows' products are pa_rows.cu's.  With few rows to a batch a run of states
// is cut into parts, so that all SMs read it, and the kernel here joins them:
// a warp to a row, whose parts' weights are made once, a lane to a part.  Up to 16
// rows of a KV head (one decoded token, some beams) go to pa_sparse_attend.cuh (one row
// to 1,500 states, 16 heads of 64 dims: 5.5 us, 8.7 by the rows kernel).
#include <math.h>

#include "pa_sparse_attend.cuh"

namespace pa {
namespace rows {

constexpr int kJoinWarps = 8;
// Up to so many rows (a sequence's tokens times a KV head's group) go to the kernel
// of the block-sparse decode, which attends to whole tables as well: its products
// take the rows as they are, where a tile has 128, and it needs no workspace.
constexpr int kFewRows = 16;

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const Args a, const float v_scale, __nv_bfloat16 *out) {
    const int lane = threadIdx.x & 31, s = blockIdx.y;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5);
    const int t = static_cast<int>(row / a.num_q_heads), hq = static_cast<int>(row - static_cast<int64_t>(t) * a.num_q_heads);
    // What the call was given is there already: the kernel before has waited for those
    // before it.
    const int first = __ldcg(a.query_start + s), end = __ldcg(a.query_start + s + 1);
    const int keys = min(max(__ldcg(a.lens + s), 0), a.max_blocks * a.block_size);
    const float scale = a.v_scales ? __ldcg(a.v_scales + hq / a.group) : v_scale;
    dependent_wait();
    if (!query_range(a, first, end) || t >= end - first) return;
    const int parts = live_parts((keys + kKeys - 1) / kKeys, a.parts);
    const int64_t at = (static_cast<int64_t>(first) + t) * a.num_q_heads + hq, rows = static_cast<int64_t>(a.num_tokens) * a.num_q_heads;
    const float2 ml = lane < parts ? __ldcg(a.part_ml + lane * rows + at) : make_float2(-INFINITY, 0.f);
    join_row<D>(ml, parts, a.part_o + at * D, rows * D, nullptr, scale, out + at * D);
}

// How a call is launched: by its sizes alone, which the workspace's size goes by too.
struct Plan {
    bool few;   // one kernel for a handful of rows
    int tiles;  // else: to a CTA
    int parts;  // of each run
};

static Plan plan(int64_t num_seqs, int64_t num_tokens, int max_query_len, int num_q_heads, int num_kv_heads, int head_dim,
                 int max_blocks, int block_size) {
    const int group = num_q_heads / num_kv_heads;
    if (static_cast<int64_t>(max_query_len) * group <= kFewRows) return {true, 0, 1};
    const int tiles = max_query_len <= tile_rows(1) / group ? 1 : 2;
    const int64_t ctas = tile_ctas(max_query_len, group, tiles) * num_kv_heads * num_seqs;
    const int blocks = static_cast<int>((static_cast<int64_t>(max_blocks) * block_size + kKeys - 1) / kKeys);
    return {false, tiles, choose_parts(ctas, blocks, tiles, head_dim, num_tokens * num_q_heads, num_seqs == 1, true)};
}

}  // namespace rows
}  // namespace pa

using namespace pa;
using namespace pa::rows;

extern "C" {

size_t pa_cross_workspace_size(int num_tokens, int num_seqs, int max_query_len, int num_q_heads, int num_kv_heads,
                               int head_dim, int max_blocks_per_seq, int block_size) {
    if (num_tokens <= 0 || num_seqs <= 0 || max_query_len <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
        num_q_heads % num_kv_heads || num_q_heads / num_kv_heads > 16 || head_dim <= 0 || max_blocks_per_seq <= 0 || block_size <= 0 ||
        static_cast<int64_t>(max_blocks_per_seq) * block_size > 0x7fffffffLL)
        return 0;
    if (max_query_len > num_tokens) max_query_len = num_tokens;
    const Plan p = plan(num_seqs, num_tokens, max_query_len, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, block_size);
    return p.parts > 1 ? workspace_bytes(p.parts, static_cast<int64_t>(num_tokens) * num_q_heads, head_dim) : 0;
}

pa_status pa_cross_attention(const void *q, const void *k_cache, const void *v_cache, const int32_t *block_tables,
                             int max_blocks_per_seq, const int32_t *state_lens, const int32_t *query_start, int num_seqs,
                             int num_tokens, int max_query_len, int num_q_heads, int num_kv_heads, int head_dim,
                             int num_blocks, int block_size, pa_kv_dtype kv_dtype, float kv_scale, const float *k_scales,
                             const float *v_scales, float softmax_scale, void *workspace, size_t workspace_bytes,
                             void *out, cudaStream_t stream) {
    clear_error();
    Args a = {};
    pa_status st = check_rows(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, num_blocks, block_size,
                              max_blocks_per_seq, kv_dtype, kv_scale, k_scales, v_scales, softmax_scale);
    if (st != PA_OK) return st;
    if (max_query_len < 0) return fail(PA_ERR_INVALID_ARG, "max_query_len %d is negative", max_query_len);
    if (num_seqs == 0 || num_tokens == 0) return PA_OK;
    if (max_query_len == 0) return fail(PA_ERR_INVALID_ARG, "max_query_len 0 with %d rows", num_tokens);
    if (max_query_len > num_tokens) max_query_len = num_tokens;
    if (!query_start) return fail(PA_ERR_INVALID_ARG, "null pointer");
    st = check_row_pointers(q, k_cache, v_cache, block_tables, state_lens, out, num_tokens, num_q_heads, head_dim);
    if (st != PA_OK) return st;
    const Plan p = plan(num_seqs, num_tokens, max_query_len, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, block_size);
    const int64_t num_rows = static_cast<int64_t>(num_tokens) * num_q_heads;
    if (p.parts > 1) {
        st = check_workspace(workspace, workspace_bytes, rows::workspace_bytes(p.parts, num_rows, head_dim), q, out,
                             static_cast<size_t>(num_rows) * head_dim * 2);
        if (st != PA_OK) return st;
    }
    unsigned int *err = device_error_word();
    if (!err) return fail(PA_ERR_CUDA, "cannot resolve the device error word");
    const bool fp8 = kv_dtype == PA_KV_FP8_E4M3;
    const int group = num_q_heads / num_kv_heads;
    if (p.few) {
        const int64_t pool_rows = static_cast<int64_t>(num_blocks) * num_kv_heads * block_size;
        CUtensorMap tk, tv;
        st = make_map(&tk, k_cache, fp8, head_dim, pool_rows, block_size);
        if (st == PA_OK) st = make_map(&tv, v_cache, fp8, head_dim, pool_rows, block_size);
        if (st != PA_OK) return st;
        sparse::Args b = {};
        b.q = static_cast<const __nv_bfloat16 *>(q);
        b.block_tables = block_tables;
        b.context_lens = state_lens;
        b.out = static_cast<__nv_bfloat16 *>(out);
        b.max_blocks = max_blocks_per_seq;
        b.num_blocks = num_blocks;
        b.num_q_heads = num_q_heads;
        b.num_kv_heads = num_kv_heads;
        b.group = group;
        b.softmax_log2 = softmax_scale * 1.4426950408889634f;
        b.kv_scale = kv_scale;
        b.k_scales = k_scales;
        b.v_scales = v_scales;
        b.err = err;
        b.wait_limit_ns = wait_limit_ns();
        b.stall_first_wait = stall_first_wait();
        b.query_start = query_start;
        b.num_tokens = num_tokens;
        b.max_query_len = max_query_len;
        const int live = max_query_len * group;
        const sparse::Spread l = sparse::spread_of_tables(static_cast<int64_t>(num_seqs) * num_kv_heads, max_blocks_per_seq,
                                                          sparse::resident_ctas(head_dim, block_size, fp8, live), live);
        return sparse::launch_any<sparse::kRows>(head_dim, block_size, fp8, tk, tv, b, num_seqs, l.splits, l.warps, stream, live);
    }
    a.block_tables = block_tables;
    a.lens = state_lens;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.group = group;
    a.num_tokens = num_tokens;
    a.num_seqs = num_seqs;
    a.max_query_len = max_query_len;
    a.softmax_log2 = softmax_scale * 1.4426950408889634f;
    a.kv_scale = kv_scale;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.parts = p.parts;
    a.query_start = query_start;
    a.err = err;
    if (p.parts == 1) {
        a.out = static_cast<__nv_bfloat16 *>(out);
    } else {
        a.part_o = static_cast<float *>(workspace);
        a.part_ml = reinterpret_cast<float2 *>(a.part_o + p.parts * num_rows * head_dim);
    }
    st = launch_rows(q, k_cache, v_cache, head_dim, fp8, a, p.tiles, tile_ctas(max_query_len, group, p.tiles), num_seqs, stream);
    if (st != PA_OK || p.parts == 1) return st;
    const int64_t join = (static_cast<int64_t>(max_query_len) * num_q_heads + kJoinWarps - 1) / kJoinWarps;
    const dim3 grid(static_cast<unsigned>(join), num_seqs);
    const float v_scale = fp8 ? kv_scale : 1.f;
    auto *to = static_cast<__nv_bfloat16 *>(out);
    return cuda_check(head_dim == 128 ? launch_dependent(join_kernel<128>, grid, kJoinWarps * 32, 0, 0, stream, a, v_scale, to)
                                      : launch_dependent(join_kernel<64>, grid, kJoinWarps * 32, 0, 0, stream, a, v_scale, to),
                      "cross attention join launch");
}

}  // extern "C"
