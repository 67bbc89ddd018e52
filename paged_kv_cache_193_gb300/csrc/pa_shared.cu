// Decode attention of a batch whose sequences share, in groups, the first pages
// of their contexts ("vLLM PagedAttention: Memory Optimization & High-Throughput
// LLM Inference Tuning", section 2: requests may point at the same physical
// pages).
//
// Two kernels.  The first takes a group's prefix once: the queries of all its
// sequences, 128 rows to a tile, against the prefix's keys (pa_rows.cu), and
// leaves each row's maximum, sum and accumulator.  The second attends to what
// each sequence has of its own, a cluster of CTAs to a (sequence, KV head)
// (pa_sparse_attend.cuh), and joins the two at its end.  It is on the SMs as
// soon as there is room beside the first's last CTAs: only its join waits for
// the prefix.
//
// A sequence that does not hold the whole prefix of its group attends to all it
// has in the second kernel.
#include "pa_sparse_attend.cuh"

namespace pa {
namespace rows {

// How a prefix's kernel is launched: by a call's sizes alone, which the workspace's
// size goes by too.
struct Plan {
    bool shared;   // or each sequence by itself
    int tiles;     // to a CTA: one where a group mostly has no more
    int64_t ctas;  // to a part and KV head: every group may have one that is not full
    int parts;
};

// A prefix's kernel costs some 6 us beside its work; up to 64 MB of prefixes, each
// counted for every sequence, are read faster than that, from the second-level cache
// but for the first time (8 KV heads of 128 dims, microseconds with and without it:
// 4 sequences of 1,024 tokens 10.0 and 7.4, 4 of 4,096 11.7 and 12.4, 32 of 1,024 in
// E4M3 11.6 and 12.7, 16 of 1,024 in bf16 10.5 and 10.3).
constexpr int64_t kShareBytes = 64000000;
static std::atomic<int64_t> g_share_bytes{kShareBytes};  // pa_test_set_share_bytes

static Plan plan(int64_t num_seqs, int num_groups, int num_q_heads, int num_kv_heads, int head_dim, int max_prefix_blocks,
                 int block_size, bool fp8) {
    const double all = static_cast<double>(num_seqs) * max_prefix_blocks * block_size * num_kv_heads * head_dim * (fp8 ? 2 : 4);
    if (num_groups == 0 || max_prefix_blocks == 0 || all <= static_cast<double>(g_share_bytes.load(std::memory_order_relaxed))) return {false, 0, 0, 0};
    const int group = num_q_heads / num_kv_heads;
    const int tiles = num_seqs <= static_cast<int64_t>(tile_rows(1) / group) * num_groups ? 1 : 2;
    const int64_t ctas = std::min(tile_ctas(num_seqs, group, tiles) + num_groups - 1, num_seqs);
    const int blocks = static_cast<int>((static_cast<int64_t>(max_prefix_blocks) * block_size + kKeys - 1) / kKeys);
    return {true, tiles, ctas, choose_parts(ctas * num_kv_heads, blocks, tiles, head_dim, num_seqs * num_q_heads, num_groups == 1, false)};
}

// How the rest is launched: at most `pages` pages behind the prefix of each of
// `num_seqs` sequences.
struct Suffix {
    bool heads;          // a warp to a KV head, not a CTA
    bool longest_first;
    int splits;          // CTAs to a sequence and KV head
};

// A CTA for every KV head costs about 3.6 us, however little it reads, so few pages
// are better read by a warp to a head (1,024 rows of up to 100 tokens: 16.1 us, 22.1
// with a CTA to each; of up to 500 43 and 29), where all CTAs are on the SMs at once
// also some more.  With as many rows as places or a few more, the longest go first
// (512 rows of up to 1,000 tokens, E4M3: 19.5 us, 28.9 in their order); who is
// longest is known for one group, whose prefix is the same for all.  Long lists are
// shared out while 512 CTAs hold them (128 rows of up to 2,000 tokens in bf16: 36.7 us
// with one, 24.0 with two, 18.7 with four; of up to 1,000 in E4M3 11.9, 13.5, 14.4),
// and to twice that when very long (512 rows of up to 4,000, longest first: 97 with
// one, 85 with two).
static Suffix suffix_launch(int64_t num_seqs, int num_groups, int num_kv_heads, bool shared, int pages, int head_dim, int block_size,
                            bool fp8, int group) {
    const int64_t rows = num_seqs * num_kv_heads;
    if (!shared)
        return {false, false, sparse::splits_of_four_warps(rows, pages, sparse::resident_ctas(head_dim, block_size, fp8, group))};
    const int at_once = fp8 && block_size == 16 ? 2 : 1;  // pages of a warp's step
    const int steps = (pages + at_once - 1) / at_once;    // of one warp
    if ((rows >= 512 && pages <= 8) || (rows >= 2048 && steps <= 16)) return {true, false, 1};
    Suffix l{false, num_groups == 1 && num_seqs > 1 && num_seqs <= sparse::kMaxSorted && pages >= 16, 1};
    if (steps >= 48)
        for (int s : {2, 4, 8})
            if (rows * s <= 512) l.splits = s;
    if (l.splits == 1 && l.longest_first && rows <= 512 && steps >= 96) l.splits = 2;
    return l;
}

pa_status check_rows(int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int num_blocks,
                     int block_size, int max_blocks, pa_kv_dtype kv_dtype, float kv_scale, const float *k_scales,
                     const float *v_scales, float softmax_scale) {
    if (num_tokens < 0) return fail(PA_ERR_INVALID_ARG, "num_tokens %d is negative", num_tokens);
    if (max_blocks > sparse::kMaxTableBlocks && static_cast<int64_t>(max_blocks) * block_size <= 0x7fffffffLL)
        max_blocks = sparse::kMaxTableBlocks;  // the choice's own limit
    pa_status st = sparse::check_select(num_seqs, num_q_heads, num_kv_heads, head_dim, num_blocks, block_size, max_blocks, 1, 0, 1);
    if (st != PA_OK) return st;
    if (kv_dtype != PA_KV_BF16 && kv_dtype != PA_KV_FP8_E4M3)
        return fail(PA_ERR_UNSUPPORTED, "kv_dtype %d", static_cast<int>(kv_dtype));
    if (!isfinite(softmax_scale) || softmax_scale <= 0.f)
        return fail(PA_ERR_INVALID_ARG, "softmax_scale must be positive and finite");
    if ((k_scales == nullptr) != (v_scales == nullptr))
        return fail(PA_ERR_INVALID_ARG, "k_scales and v_scales must both be given or both be NULL");
    if (k_scales && kv_dtype != PA_KV_FP8_E4M3)
        return fail(PA_ERR_INVALID_ARG, "per-head scales need an E4M3 cache");
    if (kv_dtype == PA_KV_FP8_E4M3 && !k_scales && !(kv_scale > 0.f && isfinite(kv_scale)))
        return fail(PA_ERR_INVALID_ARG, "fp8 kv_scale must be positive and finite");
    return PA_OK;
}

pa_status check_row_pointers(const void *q, const void *k_cache, const void *v_cache, const int32_t *block_tables,
                             const int32_t *lens, const void *out, int64_t num_tokens, int num_q_heads, int head_dim) {
    if (!q || !k_cache || !v_cache || !block_tables || !lens || !out) return fail(PA_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
        return fail(PA_ERR_INVALID_ARG, "q, k_cache, v_cache and out must be 16-byte aligned");
    const size_t bytes = static_cast<size_t>(num_tokens) * num_q_heads * head_dim * 2;
    if (out != q && overlaps(q, bytes, out, bytes)) return fail(PA_ERR_INVALID_ARG, "out overlaps q but is not q itself");
    return PA_OK;
}

pa_status check_workspace(const void *workspace, size_t got, size_t need, const void *q, const void *out, size_t row_bytes) {
    if (!workspace || got < need) return fail(PA_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace ? got : 0, need);
    if (!aligned16(workspace)) return fail(PA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    if (overlaps(workspace, need, q, row_bytes) || overlaps(workspace, need, out, row_bytes))
        return fail(PA_ERR_INVALID_ARG, "workspace overlaps q or out");
    return PA_OK;
}

}  // namespace rows
}  // namespace pa

using namespace pa;

extern "C" {

pa_status pa_test_set_share_bytes(int64_t bytes) {
    clear_error();
    rows::g_share_bytes.store(bytes < 0 ? rows::kShareBytes : bytes, std::memory_order_relaxed);
    return PA_OK;
}

size_t pa_shared_prefix_workspace_size(int num_seqs, int num_groups, int num_q_heads, int num_kv_heads, int head_dim,
                                       int block_size, int max_prefix_blocks, pa_kv_dtype kv_dtype) {
    if (num_seqs <= 0 || num_groups <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads ||
        num_q_heads / num_kv_heads > 16 || head_dim <= 0 || block_size <= 0 || max_prefix_blocks <= 0 ||
        static_cast<int64_t>(max_prefix_blocks) * block_size > 0x7fffffffLL)
        return 0;
    const rows::Plan p = rows::plan(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim, max_prefix_blocks, block_size,
                                    kv_dtype == PA_KV_FP8_E4M3);
    return rows::workspace_bytes(p.parts, static_cast<int64_t>(num_seqs) * num_q_heads, head_dim);
}

pa_status pa_shared_prefix_decode(const void *q, const void *k_cache, const void *v_cache, const int32_t *block_tables,
                                  int max_blocks_per_seq, const int32_t *context_lens, int num_seqs,
                                  const int32_t *group_start, const int32_t *prefix_blocks, int num_groups,
                                  int max_prefix_blocks, int num_q_heads, int num_kv_heads, int head_dim, int num_blocks,
                                  int block_size, pa_kv_dtype kv_dtype, float kv_scale, const float *k_scales,
                                  const float *v_scales, float softmax_scale, void *workspace, size_t workspace_bytes,
                                  void *out, cudaStream_t stream) {
    clear_error();
    pa_status st = rows::check_rows(num_seqs, num_seqs, num_q_heads, num_kv_heads, head_dim, num_blocks, block_size,
                                    max_blocks_per_seq, kv_dtype, kv_scale, k_scales, v_scales, softmax_scale);
    if (st != PA_OK) return st;
    if (num_groups < 0 || max_prefix_blocks < 0)
        return fail(PA_ERR_INVALID_ARG, "bad size (num_groups=%d, max_prefix_blocks=%d)", num_groups, max_prefix_blocks);
    if (max_prefix_blocks > max_blocks_per_seq)
        return fail(PA_ERR_INVALID_ARG, "max_prefix_blocks %d exceeds the tables' width %d", max_prefix_blocks, max_blocks_per_seq);
    if (num_groups > num_seqs)
        return fail(PA_ERR_INVALID_ARG, "%d groups of %d sequences", num_groups, num_seqs);
    if (num_seqs == 0) return PA_OK;
    st = rows::check_row_pointers(q, k_cache, v_cache, block_tables, context_lens, out, num_seqs, num_q_heads, head_dim);
    if (st != PA_OK) return st;
    const int64_t num_rows = static_cast<int64_t>(num_seqs) * num_q_heads;
    const bool fp8 = kv_dtype == PA_KV_FP8_E4M3;
    const rows::Plan p = rows::plan(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim, max_prefix_blocks, block_size, fp8);
    const bool shared = p.shared;
    if (shared) {
        if (!group_start || !prefix_blocks) return fail(PA_ERR_INVALID_ARG, "null pointer");
        st = rows::check_workspace(workspace, workspace_bytes, rows::workspace_bytes(p.parts, num_rows, head_dim), q, out,
                                   static_cast<size_t>(num_rows) * head_dim * 2);
        if (st != PA_OK) return st;
    }
    unsigned int *err = device_error_word();
    if (!err) return fail(PA_ERR_CUDA, "cannot resolve the device error word");
    const int group = num_q_heads / num_kv_heads;
    float *part_o = static_cast<float *>(workspace);
    float2 *part_ml = reinterpret_cast<float2 *>(part_o + p.parts * num_rows * head_dim);

    if (shared) {
        rows::Args a = {};
        a.block_tables = block_tables;
        a.lens = context_lens;
        a.max_blocks = max_blocks_per_seq;
        a.num_blocks = num_blocks;
        a.block_size = block_size;
        a.num_q_heads = num_q_heads;
        a.num_kv_heads = num_kv_heads;
        a.group = group;
        a.num_tokens = a.num_seqs = num_seqs;
        a.softmax_log2 = softmax_scale * 1.4426950408889634f;
        a.kv_scale = kv_scale;
        a.k_scales = k_scales;
        a.v_scales = v_scales;
        a.parts = p.parts;
        a.part_o = part_o;
        a.part_ml = part_ml;
        a.group_start = group_start;
        a.prefix_blocks = prefix_blocks;
        a.num_groups = num_groups;
        a.max_prefix_blocks = max_prefix_blocks;
        a.err = err;
        st = rows::launch_rows(q, k_cache, v_cache, head_dim, fp8, a, p.tiles, p.ctas, 1, stream);
        if (st != PA_OK) return st;
    }

    const int64_t pool_rows = static_cast<int64_t>(num_blocks) * num_kv_heads * block_size;
    CUtensorMap tk, tv;
    st = make_map(&tk, k_cache, fp8, head_dim, pool_rows, block_size);
    if (st == PA_OK) st = make_map(&tv, v_cache, fp8, head_dim, pool_rows, block_size);
    if (st != PA_OK) return st;
    sparse::Args b = {};
    b.q = static_cast<const __nv_bfloat16 *>(q);
    b.block_tables = block_tables;
    b.context_lens = context_lens;
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
    b.prefix = {group_start, prefix_blocks, num_groups, max_prefix_blocks, p.parts, part_o, part_ml, num_rows};
    // behind the prefix: of several groups, the shortest may be none
    const int pages = max_blocks_per_seq - (shared && num_groups == 1 ? max_prefix_blocks : 0);
    const rows::Suffix suffix = rows::suffix_launch(num_seqs, num_groups, num_kv_heads, shared, pages, head_dim, block_size, fp8, group);
    b.longest_first = suffix.longest_first;
    if (suffix.heads)
        return sparse::launch_any<sparse::kSuffixHeads>(head_dim, block_size, fp8, tk, tv, b, num_seqs, 1, 4, stream, group);
    return sparse::launch_any<sparse::kSuffix>(head_dim, block_size, fp8, tk, tv, b, num_seqs, suffix.splits, 4, stream, group);
}

}  // extern "C"
