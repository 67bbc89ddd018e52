// Decode attention of a batch whose sequences share, in groups, the first pages
// of their contexts ("vLLM PagedAttention: Memory Optimization & High-Throughput
// LLM Inference Tuning", section 2: requests may point at the same physical
// pages).
//
// Two kernels.  The first takes a group's prefix once: the queries of all its
// sequences, up to 128 rows to a tile, against the prefix's keys (pa_rows.cu), and
// leaves each row's maximum, sum and accumulator.  The second attends to what
// each sequence has of its own, a cluster of CTAs to a (sequence, KV head)
// (pa_sparse_attend.cuh), and joins the two at its end.  It is on the SMs as
// soon as there is room beside the first's CTAs: only its join waits for the
// prefix.  Where both have much to do the prefix takes a part of the SMs, the rest
// goes on beside it without waiting, and a third kernel joins them.
//
// A sequence that does not hold the whole prefix of its group attends to all it
// has in the second kernel.
//
// Bound: a prefix's products by the tensor cores and the chain of its softmax (64
// sequences of 64 heads over 32,768 tokens: 69 GFLOP in 55 us alone), the rest by
// memory.  Both, with up to 2,048 tokens more each: 78.2 us, where the decode that
// reads every prefix again takes 570.
#include <math.h>

#include "pa_sparse_attend.cuh"

namespace pa {
namespace rows {

// What a call's sizes say; the launches go by it.
struct Sizes {
    int64_t num_seqs;
    int num_groups, num_q_heads, num_kv_heads, head_dim, block_size, max_prefix_blocks;
    bool fp8;
    int group() const { return num_q_heads / num_kv_heads; }
    int64_t rows() const { return num_seqs * num_q_heads; }
    double page_bytes() const { return static_cast<double>(block_size) * num_kv_heads * head_dim * (fp8 ? 2 : 4); }
};

// How a prefix is taken.  The workspace's size goes by it.
struct Plan {
    bool shared;   // or each sequence by itself
    int tiles;     // to a CTA: one where a group mostly has no more
    int64_t ctas;  // to a part and KV head: every group may have one that is not full
    int parts;
};

// A prefix's kernel costs some 6 us beside its work; up to 100 MB of prefixes, each
// counted for every sequence, are read faster than that, from the second-level cache
// but for the first time, and to twice that where a group has fewer than eight sequences
// (8 KV heads of 128 dims, microseconds shared and not: 4 sequences of 1,024 tokens 10.2 and
// 7.7, 16 of 1,024 11.0 and 10.4, 16 of 2,048 12.1 and 14.3, 4 of 8,192 18.6 and 16.6, 4 of
// 16,384 23.2 and 25.5; in E4M3 32 of 1,024 14.5 and 11.6, 32 of 2,048 15.8 and 17.5, 4 of 16,384
// 24.3 and 20.1).
constexpr int64_t kShareBytes = 100000000;
static std::atomic<int64_t> g_share_bytes{kShareBytes};  // pa_test_set_share
static std::atomic<int> g_apart{-1};

static int prefix_blocks_of(const Sizes &z) {
    return static_cast<int>((static_cast<int64_t>(z.max_prefix_blocks) * z.block_size + kKeys - 1) / kKeys);
}

static Plan plan(const Sizes &z) {
    const double all = z.num_seqs * z.max_prefix_blocks * z.page_bytes();
    if (z.num_groups == 0 || z.max_prefix_blocks == 0 ||
        all <= static_cast<double>(g_share_bytes.load(std::memory_order_relaxed)) * (z.num_seqs < 8 * static_cast<int64_t>(z.num_groups) ? 2 : 1))
        return {false, 0, 0, 0};
    const int tiles = z.num_seqs <= static_cast<int64_t>(tile_rows(1) / z.group()) * z.num_groups ? 1 : 2;
    const int64_t ctas = std::min(tile_ctas(z.num_seqs, z.group(), tiles) + z.num_groups - 1, z.num_seqs);
    return {true, tiles, ctas,
            choose_parts(ctas * z.num_kv_heads, prefix_blocks_of(z), tiles, z.head_dim, z.rows(), z.num_groups == 1, false)};
}

// The prefix's parts, and one of the rest.
static size_t plan_bytes(const Sizes &z, const Plan &p) {
    return p.shared ? workspace_bytes(p.parts + 1, z.rows(), z.head_dim) : 0;
}

// A call's sizes, and how it takes its prefixes, where the tables' width is known: no prefix
// is longer than that.  The workspace may have been sized by the bound as it was given or
// by the width, so there are no more parts than either has room for.
static Sizes within_tables(Sizes z, int max_blocks) {
    z.max_prefix_blocks = std::min(z.max_prefix_blocks, max_blocks);
    return z;
}
static Plan plan(const Sizes &z, int max_blocks) {
    Plan p = plan(within_tables(z, max_blocks));
    if (p.shared && z.max_prefix_blocks > max_blocks) p.parts = std::min(p.parts, plan(z).parts);  // the longer are shared too
    return p;
}

// How the rest is launched.
struct Suffix {
    bool heads;          // a warp to a KV head, not a CTA
    bool longest_first;
    int splits, warps;   // CTAs to a sequence and KV head, and warps of a CTA
    bool apart;          // the join is a kernel of its own, and the prefix has so many parts
    int parts;
};

// A CTA for every KV head costs about 3.6 us, however little it reads, so few pages are better read
// by a warp to a head (1,024 rows of up to 100 tokens, behind 1,024: 15.2 us, 20.8 with a CTA to
// each; of up to 500 43 and 29), where all CTAs are on the SMs at once also some more.
//
// A row without its group's prefix, or of no group, has all its pages among the rest's, and a warp
// takes a microsecond to a page: under 1,536 rows a warp to a head is for tables of up to 128 pages
// (128 sequences, up to 100 tokens behind 16,384, one of them a token short of those: 1,087 us, 305
// with CTAs, and without it 46 and 45; behind 8,000 8,192 rows take 137 and 164).
//
// A bound as wide as the tables says nothing of the rest, which is then planned as if it had the
// tables to itself (64 sequences behind 32,768, up to 2,048 more, without a bound: 99 us, 204 when
// that was taken for no room, 79 with it; behind 1,024, up to 8,000 more: 170, 542 and 169), but
// for 2,048 rows and more of up to 512 pages, which a warp to a head serves whatever they are
// (1,024 sequences behind 1,024, up to 100 more: 62 us, 88 with CTAs; 256, up to 2,000 more: 194
// and 167).
//
// With as many rows as places or a few more, the longest go first (512 rows of up to 1,000 tokens,
// E4M3: 19.5 us, 28.9 in their order); who is longest is known for one group, whose prefix is the
// same for all.  Long lists are shared out while 512 CTAs hold them (128 rows of up to 2,000 tokens
// in bf16: 36.7 us with one, 24.0 with two, 18.7 with four; of up to 1,000 in E4M3 11.9, 13.5,
// 14.4), and some more when very long (with a prefix of 8,192, of up to 4,000 tokens: 512 rows
// 105.8 with one and 92.3 with two, 192 rows 53.2 with two and 48.4 with four, 128 rows 37.6 with
// four and 44.3 with eight; 512 rows of up to 2,000, behind 32,768: 79.0 with one and 91.7 with
// two).  Rows that find places at once as CTAs of eight warps have those (the same prefix, of up to
// 1,000: 128 rows 20.7 us, 22.1 by two CTAs of four warps, 26.9 by one; 32 rows in E4M3 19.5, 20.9,
// 21.3), and two of them to each of up to 2,000 (128 rows 29.1 us, 31.2 with one).
//
// The join is made apart where an estimate of both ways says so: then the prefix's CTAs
// may leave SMs to the rest's, and neither waits for the other (64 sequences, 32,768
// tokens of prefix and up to 2,048 more: 101.2 us joined by the rest's kernel, 78.6
// apart; 256 in E4M3, 2,048 and up to 512: 50.1 and 44.9; a few sequences of a few
// thousand tokens take 2 us more apart).
static Suffix suffix_launch(const Sizes &z, const Plan &p, int max_blocks) {
    const int64_t rows = z.num_seqs * z.num_kv_heads;
    // pages behind the prefix: of several groups, the shortest may be none
    const int own = max_blocks - z.max_prefix_blocks;  // 0: not known
    const int pages = p.shared && z.num_groups == 1 && own > 0 ? own : max_blocks;
    const int resident = sparse::resident_ctas(z.head_dim, z.block_size, z.fp8, z.group());
    if (!p.shared) {
        const sparse::Spread s = sparse::spread_of_tables(rows, pages, resident, z.group());
        return {false, false, s.splits, s.warps, false, 0};
    }
    const int at_once = z.fp8 && z.block_size == 16 ? 2 : 1;  // pages of a warp's step
    const int steps = (pages + at_once - 1) / at_once;        // of one warp
    const int mode = g_apart.load(std::memory_order_relaxed);
    const bool lone = rows >= 1536 || max_blocks <= 128;
    if ((rows >= 512 && pages <= 8 && lone) || (z.num_groups == 1 && own == 0 && rows >= 2048 && pages <= 512))
        // joined by these, unless a test asks for the other way
        return {true, false, 1, 4, mode == 1, mode == 1 ? std::min(p.parts, kMaxParts - 1) : p.parts};
    Suffix l{false, z.num_groups == 1 && z.num_seqs > 1 && z.num_seqs <= sparse::kMaxSorted && pages >= 16, 1, 4, false, p.parts};
    const int64_t wide = sparse::places_of_eight_warps(resident, z.group());
    if (rows <= wide && pages >= 12 && (steps < 160 || rows * 4 <= wide)) {
        l.warps = 8;
        for (int s : {2, 4, 8})
            if (rows * s <= wide && steps >= 48 * s) l.splits = s;
    } else if (steps >= 48)
        for (int s : {2, 4, 8})
            if (rows * s <= (steps >= 160 ? 512 + 1024 / s : 512)) l.splits = s;

    const int64_t ctas = p.ctas * z.num_kv_heads, places = (p.tiles == 1 ? 2 : 1) * kSms;
    const int blocks = prefix_blocks_of(z);
    const double average = z.num_groups == 1 ? 1.0 : 0.6;  // of runs of unlike lengths, beside the longest
    auto one = [&](int parts) { return cta_time(blocks_per_part(blocks, parts), p.tiles, z.head_dim); };
    auto waves = [&](int parts) { return std::ceil(static_cast<double>(ctas) * parts / places); };
    const double alone = waves(p.parts) * one(p.parts) * average;
    // Half of the pages that the tables have room for, at 6.2 TB/s; many short lists go
    // a little slower.  Tables may be far wider than what they hold, and a prefix that is cut
    // for a rest of that length ends long after the real one, so a rest of several times the
    // prefix's own time counts for as much as that (64 sequences behind 32,768 tokens, up to
    // 2,048 more, tables for 131,072: 92 us, 376 else; where there is so much, 64 sequences
    // behind 1,024, up to 8,000 more: 170.7 and 169.0).
    double rest = z.num_seqs * own * 0.5 * z.page_bytes() / 6.2e6 * (pages < 64 ? 1.3 : 1.0);
    if (rest > 4 * alone) rest = alone;
    const double together = alone + join_time(p.parts, z.head_dim, z.rows()) + rest;
    double least = INFINITY;
    for (int parts = 1; parts <= p.parts && parts < kMaxParts; ++parts) {
        const double cost = std::max(waves(parts) * one(parts), ctas * parts * one(parts) * average / places + rest) +
                            join_time(parts + 1, z.head_dim, z.rows()) + 3.0;
        if (cost < least) {
            least = cost;
            l.parts = parts;
        }
    }
    l.apart = mode == 1 || (mode < 0 && least < together);
    // A warp to a head (1,600 rows of up to 200 and 300 tokens, E4M3, apart: 30.7 and 30.8 us,
    // 32.5 and 35.7 with a CTA to each; of up to 200 and 300 in bf16 31.6 and 39.4, 33.5 and 37.8;
    // 2,048 rows of up to 512, E4M3, 45.8 and 44.9, but joined by them 49.0 and 50.1).
    if (rows >= 1536 && steps <= (l.apart ? 13 : 16) && lone) {
        l.heads = true;
        l.longest_first = false;
        l.splits = 1;
        l.warps = 4;
    }
    if (!l.apart) l.parts = p.parts;
    return l;
}

constexpr int kJoinWarps = 8;

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
    join_prefix_kernel(const sparse::Args a, const int num_seqs, const int block_size, const float v_scale) {
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5), seq = row / a.num_q_heads;
    const int s = static_cast<int>(seq), hq = static_cast<int>(row - seq * a.num_q_heads);
    // What the call was given is there already: the prefix's kernel has waited for those
    // before it.
    int parts = 0;
    float scale = v_scale;
    if (seq < num_seqs) {
        const int skip = sparse::shared_pages(a.prefix, s, min(__ldcg(a.context_lens + s), a.max_blocks * block_size), block_size);
        if (skip) parts = live_parts((skip * block_size + kKeys - 1) / kKeys, a.prefix.parts);
        if (a.v_scales) scale = __ldcg(a.v_scales + hq / a.group);
    }
    dependent_wait();
    if (seq >= num_seqs) return;
    const float2 ml = lane < parts ? __ldcg(a.prefix.ml + lane * a.prefix.rows + row)
                                   : lane == 31 ? __ldcg(a.prefix.rest_ml + row) : make_float2(-INFINITY, 0.f);
    join_row<D>(ml, parts, a.prefix.o + row * D, a.prefix.rows * D, a.prefix.rest_o + row * D,
                scale, a.out + row * D);
}

pa_status check_rows(int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int num_blocks,
                     int block_size, int max_blocks, pa_kv_dtype kv_dtype, float kv_scale, const float *k_scales,
                     const float *v_scales, float softmax_scale) {
    if (num_tokens < 0) return fail(PA_ERR_INVALID_ARG, "num_tokens %d is negative", num_tokens);
    const bool wide = max_blocks > sparse::kMaxTableBlocks && static_cast<int64_t>(max_blocks) * block_size <= 0x7fffffffLL;
    pa_status st = sparse::check_select(num_seqs, num_q_heads, num_kv_heads, head_dim, num_blocks, block_size,
                                        wide ? sparse::kMaxTableBlocks : max_blocks, 1, 0, 1);  // the choice's own limit
    if (st != PA_OK) return st;
    if (static_cast<int64_t>(max_blocks) * block_size > 0x7fff0000LL)  // room to count past the end in blocks of keys
        return fail(PA_ERR_UNSUPPORTED, "tables for more than 2^31 - 2^16 tokens");
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

pa_status pa_test_set_share(int64_t bytes, int apart) {
    clear_error();
    if (apart < -1 || apart > 1) return fail(PA_ERR_INVALID_ARG, "apart %d (-1, 0 or 1)", apart);
    rows::g_share_bytes.store(bytes < 0 ? rows::kShareBytes : bytes, std::memory_order_relaxed);
    rows::g_apart.store(apart, std::memory_order_relaxed);
    return PA_OK;
}

size_t pa_shared_prefix_workspace_size(int num_seqs, int num_groups, int num_q_heads, int num_kv_heads, int head_dim,
                                       int block_size, int max_prefix_blocks, pa_kv_dtype kv_dtype) {
    if (num_seqs <= 0 || num_groups <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads ||
        num_q_heads / num_kv_heads > 16 || (head_dim != 64 && head_dim != 128) || block_size <= 0 || max_prefix_blocks <= 0 ||
        static_cast<int64_t>(max_prefix_blocks) * block_size > 0x7fffffffLL)
        return 0;
    const rows::Sizes z{num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim, block_size, max_prefix_blocks, kv_dtype == PA_KV_FP8_E4M3};
    return rows::plan_bytes(z, rows::plan(z));
}

int pa_shared_prefix_launches(int num_seqs, int num_groups, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                              int max_blocks_per_seq, int max_prefix_blocks, pa_kv_dtype kv_dtype) {
    if (num_seqs <= 0) return 0;
    if (pa_shared_prefix_workspace_size(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim, block_size, max_prefix_blocks,
                                        kv_dtype) == 0)
        return 1;
    const rows::Sizes z{num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim, block_size, max_prefix_blocks, kv_dtype == PA_KV_FP8_E4M3};
    const rows::Plan p = rows::plan(z, max_blocks_per_seq);
    return !p.shared ? 1 : rows::suffix_launch(rows::within_tables(z, max_blocks_per_seq), p, max_blocks_per_seq).apart ? 3 : 2;
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
    if (static_cast<int64_t>(max_prefix_blocks) * block_size > 0x7fffffffLL)
        return fail(PA_ERR_UNSUPPORTED, "prefixes of more than 2^31 - 1 tokens");
    if (num_groups > num_seqs)
        return fail(PA_ERR_INVALID_ARG, "%d groups of %d sequences", num_groups, num_seqs);
    if (num_seqs == 0) return PA_OK;
    st = rows::check_row_pointers(q, k_cache, v_cache, block_tables, context_lens, out, num_seqs, num_q_heads, head_dim);
    if (st != PA_OK) return st;
    const bool fp8 = kv_dtype == PA_KV_FP8_E4M3;
    const rows::Sizes given{num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim, block_size, max_prefix_blocks, fp8};
    const rows::Plan p = rows::plan(given, max_blocks_per_seq);
    const rows::Sizes z = rows::within_tables(given, max_blocks_per_seq);
    const rows::Suffix l = rows::suffix_launch(z, p, max_blocks_per_seq);
    const int64_t num_rows = z.rows();
    if (p.shared) {
        if (!group_start || !prefix_blocks) return fail(PA_ERR_INVALID_ARG, "null pointer");
        st = rows::check_workspace(workspace, workspace_bytes, rows::plan_bytes(z, p), q, out,
                                   static_cast<size_t>(num_rows) * head_dim * 2);
        if (st != PA_OK) return st;
    }
    unsigned int *err = device_error_word();
    if (!err) return fail(PA_ERR_CUDA, "cannot resolve the device error word");
    const int group = z.group();
    // the prefix's parts, then the rest's; all their (m, l) behind all their o
    float *part_o = static_cast<float *>(workspace);
    float2 *part_ml = reinterpret_cast<float2 *>(part_o + (l.parts + 1) * num_rows * head_dim);

    if (p.shared) {
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
        a.parts = l.parts;
        a.part_o = part_o;
        a.part_ml = part_ml;
        a.group_start = group_start;
        a.prefix_blocks = prefix_blocks;
        a.num_groups = num_groups;
        a.max_prefix_blocks = z.max_prefix_blocks;
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
    b.longest_first = l.longest_first;
    b.prefix = {group_start, prefix_blocks, num_groups, z.max_prefix_blocks, l.parts, part_o, part_ml, num_rows, nullptr, nullptr};
    if (l.apart) {
        b.prefix.rest_o = part_o + l.parts * num_rows * head_dim;
        b.prefix.rest_ml = part_ml + l.parts * num_rows;
    }
    st = l.heads ? sparse::launch_any<sparse::kSuffixHeads>(head_dim, block_size, fp8, tk, tv, b, num_seqs, 1, 4, stream, group)
                 : sparse::launch_any<sparse::kSuffix>(head_dim, block_size, fp8, tk, tv, b, num_seqs, l.splits, l.warps, stream, group);
    if (st != PA_OK || !l.apart) return st;
    const dim3 grid(static_cast<unsigned>((num_rows + rows::kJoinWarps - 1) / rows::kJoinWarps));
    auto *join = head_dim == 128 ? rows::join_prefix_kernel<128> : rows::join_prefix_kernel<64>;
    return cuda_check(launch_dependent(join, grid, rows::kJoinWarps * 32, 0, 0, stream, b, num_seqs, block_size, fp8 ? kv_scale : 1.f),
                      "shared prefix join launch");
}

}  // extern "C"
