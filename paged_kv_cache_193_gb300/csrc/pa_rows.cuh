// Attention of many query rows to one run of cached pages on the tcgen05
// tensor cores: what cross attention and the shared part of a prefix-sharing
// batch's decode have in common.  Here the parts that both sides of a launch
// agree on; the kernel is in pa_rows.cu.
//
// Rows are (token, query head of one KV head) pairs, up to 128 to a tile; a run of
// keys may be cut into parts, each with its own
//   m = max_t s_t (or what the kernel takes for it), l = sum_t 2^(s_t - m),
//   o = sum_t 2^(s_t - m) V[t],   s_t = softmax_scale * log2(e) * q . K[t],
// which join as M = max m, sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p.
#pragma once

#include <math.h>

#include <algorithm>

#include "pa_launch.cuh"

namespace pa {
namespace rows {

constexpr int kSms = 152;
constexpr int kRows = 128;     // rows of a product (lanes of tensor memory)
constexpr int kKeys = 64;      // keys of a block
constexpr int kMaxParts = 32;  // of a run of keys
// A part has at least so many blocks: its start and end cost about as much.
constexpr int kLeastBlocks = 4;

// Query rows of a tile, for CTAs of one or of two.
__host__ __device__ constexpr int tile_rows(int tiles) { return tiles == 1 ? kRows / 2 : kRows; }

// Blocks of each part of a run of `blocks`; parts from ceil(blocks / that) on
// have none, and nothing is written for them.
__host__ __device__ __forceinline__ int blocks_per_part(int blocks, int parts) {
    const int even = (blocks + parts - 1) / parts;
    return even > kLeastBlocks ? even : kLeastBlocks;
}
__host__ __device__ __forceinline__ int live_parts(int blocks, int parts) {
    const int each = blocks_per_part(blocks, parts);
    return (blocks + each - 1) / each;
}

// Floats of the parts: [parts][num_tokens * num_q_heads] of (head_dim, and m, l).
inline size_t workspace_bytes(int parts, int64_t num_rows, int head_dim) {
    return static_cast<size_t>(parts) * num_rows * (head_dim + 2) * sizeof(float);
}

struct Args {
    const int32_t *block_tables;
    const int32_t *lens;  // tokens of each sequence
    int max_blocks, num_blocks, block_size;
    int num_q_heads, num_kv_heads, group;
    int num_tokens, num_seqs;
    int max_query_len;   // cross attention: rows of a sequence, at most
    int tile_tokens;     // of a tile's rows
    float softmax_log2;  // softmax_scale * log2(e)
    float kv_scale;      // E4M3: one scale, or one of K and V for each head
    const float *k_scales, *v_scales;
    uint64_t wait_limit_ns;
    int stall_first_wait;
    int parts;
    __nv_bfloat16 *out;  // one part: the result goes here
    float *part_o;       // several, or a prefix: [parts][rows][head_dim]
    float2 *part_ml;     // [parts][rows]
    // cross attention: sequence s's rows are tokens query_start[s] .. query_start[s + 1] - 1
    const int32_t *query_start;
    int sorted;  // the longest runs first (found by the launch)
    // shared prefix: group g's sequences are group_start[g] .. group_start[g + 1] - 1
    const int32_t *group_start;
    const int32_t *prefix_blocks;
    int num_groups, max_prefix_blocks;
    unsigned int *err;
};

// CTAs of `tiles` tiles (1 or 2, which read the same stages) for `tokens` tokens of
// a KV head's group.
inline int64_t tile_ctas(int64_t tokens, int group, int tiles) {
    const int each = tiles * (tile_rows(tiles) / group);
    return (tokens + each - 1) / each;
}

// Estimates in microseconds: of a CTA, and of the parts' way through memory.
double cta_time(int blocks, int tiles, int head_dim);
double join_time(int parts, int head_dim, int64_t num_rows);

// Into how many parts to cut runs of up to `blocks` blocks for `ctas` CTAs to a part;
// `even`: all runs are as long as that; `direct`: one part needs no joining.
int choose_parts(int64_t ctas, int blocks, int tiles, int head_dim, int64_t num_rows, bool even, bool direct);

// Whether `first` .. `end` - 1 is a range of the tokens, and no longer than it may be.
__device__ __forceinline__ bool query_range(const Args &a, int first, int end) {
    return first >= 0 && end >= first && end <= a.num_tokens && end - first <= a.max_query_len;
}

// Joins the parts of one row and writes it: by a warp whose lane p has part p's
// (m, l), and whose last lane has those of `rest` (or of part 31, or none); part p's
// o is at o + p * stride.  Fewer than 32 parts with a rest.  Loads past the first-level
// cache: a part may be of the kernel before the one before.
template <int D>
__device__ __forceinline__ void join_row(float2 ml, int parts, const float *o, int64_t stride, const float *rest,
                                         float v_scale, __nv_bfloat16 *out) {
    constexpr int E = D / 32;  // head dims of a lane
    const int lane = threadIdx.x & 31;
    float top = ml.x;
#pragma unroll
    for (int d = 16; d; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    // a part that saw no finite score is left out, one with a NaN in its sum keeps it
    float f = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : ml.y) : fast_exp2(ml.x - top);
    float sum = f != 0.f ? f * ml.y : 0.f;
#pragma unroll
    for (int d = 16; d; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    f *= sum != 0.f ? v_scale / sum : 0.f;
    dependent_release();
    float acc[E] = {};
    auto add = [&](const float *from, float w) {
        float x[E];
        if constexpr (E == 4)
            *reinterpret_cast<float4 *>(x) = __ldcg(reinterpret_cast<const float4 *>(from + lane * E));
        else
            *reinterpret_cast<float2 *>(x) = __ldcg(reinterpret_cast<const float2 *>(from + lane * E));
        if (w != 0.f)  // an empty part's accumulator may be anything
#pragma unroll
            for (int i = 0; i < E; ++i) acc[i] += w * x[i];
    };
    if (rest) add(rest, __shfl_sync(0xffffffffu, f, 31));
#pragma unroll 4
    for (int p = 0; p < parts; ++p) add(o + p * stride, __shfl_sync(0xffffffffu, f, p));
    __nv_bfloat16 *to = out + lane * E;
    if constexpr (E == 4)
        *reinterpret_cast<uint2 *>(to) = make_uint2(pack2<false>(acc[0], acc[1]), pack2<false>(acc[2], acc[3]));
    else
        *reinterpret_cast<uint32_t *>(to) = pack2<false>(acc[0], acc[1]);
}

// Checks of arguments, for both (pa_shared.cu).
pa_status check_rows(int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int num_blocks,
                     int block_size, int max_blocks, pa_kv_dtype kv_dtype, float kv_scale, const float *k_scales,
                     const float *v_scales, float softmax_scale);
pa_status check_row_pointers(const void *q, const void *k_cache, const void *v_cache, const int32_t *block_tables,
                             const int32_t *lens, const void *out, int64_t num_tokens, int num_q_heads, int head_dim);
pa_status check_workspace(const void *workspace, size_t got, size_t need, const void *q, const void *out, size_t row_bytes);

// Attention of `a`'s rows (q bf16 [num_tokens][num_q_heads][head_dim]) over the grid's
// (tile or two, part), KV head, and sequence (1 for a shared prefix: the tiles of all groups lie
// one after the other).
pa_status launch_rows(const void *q, const void *k_cache, const void *v_cache, int head_dim, bool fp8, Args &a,
                      int tiles, int64_t ctas, int seqs, cudaStream_t stream);

}  // namespace rows
}  // namespace pa
