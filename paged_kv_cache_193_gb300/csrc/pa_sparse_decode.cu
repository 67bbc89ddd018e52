// Entry points of the block-sparse decode: attention over a given list, and
// the choice and the attention in one kernel.
#include "pa_sparse_attend.cuh"

namespace pa {
namespace sparse {

struct Call {
    const void *q, *k_cache, *v_cache;
    const int32_t *block_tables, *context_lens;
    int max_blocks, num_rows, num_q_heads, num_kv_heads, head_dim, num_blocks, block_size, top_k;
    pa_kv_dtype kv_dtype;
    float kv_scale, softmax_scale;
    const float *k_scales, *v_scales;
    int splits;
    const int32_t *selected, *counts;
    void *out;
};

static pa_status check_attend(const Call &c) {
    if (c.kv_dtype != PA_KV_BF16 && c.kv_dtype != PA_KV_FP8_E4M3)
        return fail(PA_ERR_UNSUPPORTED, "kv_dtype %d", static_cast<int>(c.kv_dtype));
    if (!isfinite(c.softmax_scale) || c.softmax_scale <= 0.f)
        return fail(PA_ERR_INVALID_ARG, "softmax_scale must be positive and finite");
    if ((c.k_scales == nullptr) != (c.v_scales == nullptr))
        return fail(PA_ERR_INVALID_ARG, "k_scales and v_scales must both be given or both be NULL");
    if (c.k_scales && c.kv_dtype != PA_KV_FP8_E4M3)
        return fail(PA_ERR_INVALID_ARG, "per-head scales need an E4M3 cache");
    if (c.kv_dtype == PA_KV_FP8_E4M3 && !c.k_scales && !(c.kv_scale > 0.f && isfinite(c.kv_scale)))
        return fail(PA_ERR_INVALID_ARG, "fp8 kv_scale must be positive and finite");
    if (c.splits != 0 && c.splits != 1 && c.splits != 2 && c.splits != 4 && c.splits != 8)
        return fail(PA_ERR_INVALID_ARG, "splits %d (supported: 0 = chosen here, 1, 2, 4, 8)", c.splits);
    return PA_OK;
}

static pa_status check_pointers(const Call &c) {
    if (!c.q || !c.k_cache || !c.v_cache || !c.block_tables || !c.context_lens || !c.selected ||
        !c.counts || !c.out)
        return fail(PA_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(c.q) || !aligned16(c.k_cache) || !aligned16(c.v_cache) || !aligned16(c.out))
        return fail(PA_ERR_INVALID_ARG, "q, k_cache, v_cache and out must be 16-byte aligned");
    const size_t bytes = static_cast<size_t>(c.num_rows) * c.num_q_heads * c.head_dim * 2;
    if (c.out != c.q && overlaps(c.q, bytes, c.out, bytes))
        return fail(PA_ERR_INVALID_ARG, "out overlaps q but is not q itself");
    return PA_OK;
}

// How a (row, KV head)'s pages are shared out.
struct Launch {
    int warps;   // to a CTA
    int splits;  // CTAs to a cluster
    bool longest_first;
};

// Four warps to a CTA: the most CTAs whose clusters are all resident at once and
// whose warps have a page each.  An eighth of the CTAs' places is kept back:
// clusters of three, six or eight leave some of a GPC's places empty (8 rows of
// 8 heads, 16 queries each, 128K tokens: 62 us with 6, 71 with 4, 85 with 8).
// Short lists are not shared out, or little (152 rows of 8 pages 4.8 us, 5.3 with two
// CTAs, of 16 query heads 5.4 and 7.8; 72 rows of 24 pages 6.1 with two, 6.7 with six).
static int splits_of_four_warps(int64_t rows, int pages, int resident) {
    const int most = pages < 16 ? 1 : pages < 32 && rows >= 48 ? 2 : 8;
    int splits = 1;
    for (int s : {2, 3, 4, 6, 8})
        if (s <= most && rows * s <= resident * kSms * 7 / 8 && pages >= 4 * s) splits = s;
    return splits;
}

// The kernel that chooses takes CTAs of eight warps while a CTA for every row
// and KV head is resident (up to 8 query heads): half the cluster for the same
// warps, and most of a choice's steps are waits for the whole cluster.
// Measured, 4 against 8 warps, each at its best: 8 rows of 128K tokens 30 and 23
// us, 64 of 128K 57 and 55, 256 of 1K-8K 33 and 30, 272 at head dim 64 16 and 14.
// Clusters of three and six of them, and of eight beyond half of the places,
// measured slower than the next smaller size (32 of 8K: 18 us with 8, 15 with 4),
// clusters of sixteen slower than of eight (8 rows of 128K: 30 us, 24 with eight).
// In clusters of two all places can be taken, in clusters of four not quite (76
// rows of 375 pages, top 128, 304 CTAs on 304 places: 32.8 us, 27.7 in clusters of
// two; 72 rows 23.3 and 26.8).
// Rows of few pages take one CTA, which needs no cluster's barriers (48 rows of 125
// pages, top 24: 8.1 us, 10.0 with two; 96 of 157: 11.7 and 14.5).  Clusters of two
// pay from some 800 pages on (96 rows of 625, top 64: 21.2 us with one CTA, 26.5
// with two; 136 of 1000, top 128: 38.6 and 37.2, of 2500, top 192: 62.5 and 56.1).
// Where four do not fit, six of four warps fill the SMs better for long rows, or
// for lists that are long beside them (96 rows of 2500 pages, top 192: 43.8 us, 47.6
// with two of eight warps; of 375, top 128: 28.0, 30.3 with one; of 94, top 24, one:
// 10.8 and 12.8), but not where only three CTAs of four warps fit an SM (72 rows of
// 1000 pages of 32 bf16 tokens, top 128: 37.3, 35.4 with two of eight warps).
static Launch chosen_launch(const Call &c, int group, int resident) {
    const int64_t rows = static_cast<int64_t>(c.num_rows) * c.num_kv_heads;
    Launch l{4, 1, false};
    int places = resident;
    if (group <= 8 && rows <= resident / 2 * kSms) {
        l.warps = 8;
        places = resident / 2;
        const int pages = std::max(c.top_k, c.max_blocks / 4);
        const int64_t room = static_cast<int64_t>(places) * kSms;
        if (rows * 2 <= room && c.max_blocks >= 800) l.splits = 2;
        if (rows * 4 <= room * 19 / 20 && pages >= 32) l.splits = 4;
        if (rows * 8 <= room / 2 && pages >= 64) l.splits = 8;
        const bool long_list = c.top_k >= 48 && c.top_k >= c.max_blocks / 8;
        if (l.splits <= 2 && resident >= 4 && rows * 6 <= resident * kSms * 19 / 20 && (c.max_blocks >= 800 || long_list)) {
            l = {4, 6, false};
            places = resident;
        }
    } else {
        l.splits = splits_of_four_warps(rows, c.top_k, resident);
        // as above (16 query heads: 192 rows of 250 pages, top 32: 20.4 us with one, 23.1
        // with two; 72 of 94, top 24: 13.1, 14.3 with six)
        if ((l.splits == 2 && c.max_blocks < 800) || (rows >= 48 && std::max(c.top_k, c.max_blocks / 4) < 32)) l.splits = 1;
    }
    while (c.max_blocks > kMaxKeys * l.splits) ++l.splits;  // at most 8, by the limit on the table
    // With a few more CTAs than places, and rows that few threads can sort, the
    // longest go first, so that the last to start are the shortest (80 rows of 8
    // heads, 2K-32K tokens, 640 CTAs on 608 places: 144 us, 159 in their order; 512
    // of 16 query heads on 456: 72 and 76).  With more, rows in any order spread
    // the choices over the time better (800 on 608, E4M3: 87 us, 92 longest first).
    const int64_t ctas = rows * l.splits, room = static_cast<int64_t>(places) * kSms;
    l.longest_first = c.num_rows > 1 && c.num_rows <= kMaxSorted && ctas > room && ctas <= room + room / 4;
    return l;
}

// `select`: choose the pages in the same kernel; otherwise the list is there.
static pa_status run_attend(const Call &c, const SelectArgs *select, cudaStream_t stream) {
    const bool fp8 = c.kv_dtype == PA_KV_FP8_E4M3;
    const int64_t pool_rows = static_cast<int64_t>(c.num_blocks) * c.num_kv_heads * c.block_size;
    CUtensorMap tk, tv;
    pa_status st = make_map(&tk, c.k_cache, fp8, c.head_dim, pool_rows, c.block_size);
    if (st != PA_OK) return st;
    st = make_map(&tv, c.v_cache, fp8, c.head_dim, pool_rows, c.block_size);
    if (st != PA_OK) return st;
    unsigned int *err = device_error_word();
    if (!err) return fail(PA_ERR_CUDA, "cannot resolve the device error word");
    Args a;
    a.q = static_cast<const __nv_bfloat16 *>(c.q);
    a.block_tables = c.block_tables;
    a.context_lens = c.context_lens;
    a.selected = c.selected;
    a.counts = c.counts;
    a.out = static_cast<__nv_bfloat16 *>(c.out);
    a.max_blocks = c.max_blocks;
    a.num_blocks = c.num_blocks;
    a.num_q_heads = c.num_q_heads;
    a.num_kv_heads = c.num_kv_heads;
    a.group = c.num_q_heads / c.num_kv_heads;
    a.top_k = c.top_k;
    a.softmax_log2 = c.softmax_scale * 1.4426950408889634f;
    a.kv_scale = c.kv_scale;
    a.k_scales = c.k_scales;
    a.v_scales = c.v_scales;
    a.err = err;
    a.wait_limit_ns = wait_limit_ns();
    a.stall_first_wait = stall_first_wait();
    const int64_t rows = static_cast<int64_t>(c.num_rows) * c.num_kv_heads;
    const int resident = resident_ctas(c.head_dim, c.block_size, fp8, a.group);
    if (select) {
        a.select = *select;
        const Launch l = chosen_launch(c, a.group, resident);
        a.longest_first = l.longest_first;
        return launch_chosen(c.head_dim, c.block_size, fp8, tk, tv, a, c.num_rows, l.splits, l.warps, stream);
    }
    const int splits = c.splits ? c.splits : splits_of_four_warps(rows, c.top_k, resident);
    return launch_any<false>(c.head_dim, c.block_size, fp8, tk, tv, a, c.num_rows, splits, 4, stream);
}

}  // namespace sparse
}  // namespace pa

using namespace pa;
using namespace pa::sparse;

extern "C" {

pa_status pa_sparse_decode(const void *q, const void *k_cache, const void *v_cache,
                           const int32_t *block_tables, int max_blocks_per_seq,
                           const int32_t *context_lens, int num_rows, int num_q_heads,
                           int num_kv_heads, int head_dim, int num_blocks, int block_size,
                           pa_kv_dtype kv_dtype, float kv_scale, const float *k_scales,
                           const float *v_scales, float softmax_scale, const int32_t *selected,
                           const int32_t *counts, int top_k, int splits, void *out,
                           cudaStream_t stream) {
    clear_error();
    const Call c{q, k_cache, v_cache, block_tables, context_lens, max_blocks_per_seq, num_rows,
                 num_q_heads, num_kv_heads, head_dim, num_blocks, block_size, top_k, kv_dtype,
                 kv_scale, softmax_scale, k_scales, v_scales, splits, selected, counts, out};
    pa_status st = check_select(num_rows, num_q_heads, num_kv_heads, head_dim, num_blocks, block_size,
                                max_blocks_per_seq, top_k, 0, 1);
    if (st == PA_OK) st = check_attend(c);
    if (st != PA_OK) return st;
    if (num_rows == 0) return PA_OK;
    st = check_pointers(c);
    return st == PA_OK ? run_attend(c, nullptr, stream) : st;
}

pa_status pa_sparse_attend(const void *q, const void *k_cache, const void *v_cache,
                           const int8_t *summary, const int8_t *exponents,
                           const int32_t *block_tables, int max_blocks_per_seq,
                           const int32_t *context_lens, int num_rows, int num_q_heads,
                           int num_kv_heads, int head_dim, int num_blocks, int block_size,
                           pa_kv_dtype kv_dtype, float kv_scale, const float *k_scales,
                           const float *v_scales, float softmax_scale, int top_k, int sink_blocks,
                           int recent_blocks, int32_t *selected, int32_t *counts, void *out,
                           cudaStream_t stream) {
    clear_error();
    const Call c{q, k_cache, v_cache, block_tables, context_lens, max_blocks_per_seq, num_rows,
                 num_q_heads, num_kv_heads, head_dim, num_blocks, block_size, top_k, kv_dtype,
                 kv_scale, softmax_scale, k_scales, v_scales, 0, selected, counts, out};
    pa_status st = check_select(num_rows, num_q_heads, num_kv_heads, head_dim, num_blocks, block_size,
                                max_blocks_per_seq, top_k, sink_blocks, recent_blocks);
    if (st == PA_OK) st = check_attend(c);
    if (st != PA_OK) return st;
    if (num_rows == 0) return PA_OK;
    st = check_pointers(c);
    if (st != PA_OK) return st;
    if (!summary || !exponents) return fail(PA_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(summary)) return fail(PA_ERR_INVALID_ARG, "summary must be 16-byte aligned");
    const SelectArgs sel = select_args(q, summary, exponents, block_tables, max_blocks_per_seq, context_lens,
                                       num_q_heads, num_kv_heads, num_blocks, block_size, top_k, sink_blocks,
                                       recent_blocks, selected, counts);
    return run_attend(c, &sel, stream);
}

}  // extern "C"
