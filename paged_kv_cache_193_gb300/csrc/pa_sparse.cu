// Which pages a decode step attends to: int8 bounds of every full page's keys
// (block summary), and the choice of the pages with the largest estimate of a
// bound of q . k (sparse select).  The pages motivate contexts of 128K tokens ("vLLM
// PagedAttention Optimization: Complete Step-by-Step Tuning Guide", Step 1)
// and attend to all of them; attending to a chosen part is this library's own.
//
// Mathematics.  For a page's keys k_t (t over its tokens) let hi_d = max_t
// k_t,d and lo_d = min_t k_t,d.  Then for any query q,
//   q . k_t <= sum_d max(q_d hi_d, q_d lo_d).
// hi, lo and q are held as whole numbers of at most 127 times a power of two
// shared by the page and head (by the query head), so the score is a whole
// number, the sum has no rounding and no order, and two pages compare the
// same way on any machine.  Eight bits with a shared power of two are coarse
// (steps of 1/64 to 1/127 of the largest value) and rounded to the nearest, not
// outward: with u_k and u_q the two units, the score is within
//   sum_d (u_k |q_d| + u_q max(|hi_d|, |lo_d|) + u_k u_q / 2) / 2
// of the bound (of values in the exponents' range), and below it about as often
// as above.  It ranks pages and bounds nothing.  Of 128 of 2,048 pages that the
// bound itself would choose it finds 97% on normal keys, 90% where four dims are
// 15 times the others (69% for the worst of 1,280 queries), 84% where two are 50
// times them (36%): the largest dim sets the unit of all.
#include "pa_sparse_select.cuh"

namespace pa {
namespace sparse {

// ---------------------------------------------------------------------------
// block summary
// ---------------------------------------------------------------------------

struct SummaryArgs {
    const uint8_t *k_cache;
    const int32_t *slots;
    int8_t *summary;    // [num_blocks][num_kv_heads][2][head_dim]: largest, least
    int8_t *exponents;  // [num_blocks][num_kv_heads]
    int64_t num_slots;
    int num_tokens, num_kv_heads;
    int per_cta;  // slots that a CTA looks at
    unsigned int *err;
};

constexpr int kSummarySlots = 16;  // looked at by a CTA, at most
constexpr int kSummaryWarps = 8;

// A CTA looks at up to 16 slots, for 8 of the heads; each of its warps takes
// (completed page, head) items in turn.  A lane reads 16-byte pieces of the page's rows, all before
// the first is used, and keeps their largest and least as packed bf16; lanes
// that hold the same head dims then join theirs, the lower half of the warp
// the largest and the upper half the least.  An E4M3 code in the upper byte of
// a bf16 is finite and keeps the codes' order (both are sign and magnitude),
// so codes are compared as they are; the code of NaN comes out as the largest
// or the least, and bf16 NaNs pass through their maximum and minimum.
//
// Bound: latency (the slots, then the page, then the joins) up to some
// thousand pages, the memory above.
template <int D, int BS, bool FP8>
__global__ void __launch_bounds__(kSummaryWarps * 32) summary_kernel(const SummaryArgs a) {
    using T = __nv_bfloat162;
    constexpr int ELEM = FP8 ? 1 : 2;
    constexpr int EPL = 16 / ELEM;  // elements of a lane's piece
    constexpr int LPR = D / EPL;    // lanes to a row
    constexpr int RPL = 32 / LPR;   // rows per load of the warp
    constexpr int LOADS = BS / RPL;
    constexpr int PAIRS = EPL / 2;
    auto pair = [](uint32_t w) { return *reinterpret_cast<const T *>(&w); };
    auto bits = [](const T &x) { return *reinterpret_cast<const uint32_t *>(&x); };
    dependent_wait();
    dependent_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int token0 = blockIdx.x * a.per_cta;
    int32_t slot = lane < min(a.per_cta, a.num_tokens - token0) ? a.slots[token0 + lane] : -1;
    if (slot >= a.num_slots) {
        if (warp == 0 && blockIdx.y == 0) set_device_error(a.err, PA_DEVERR_BAD_SLOT);
        slot = -1;
    }
    const uint32_t ends = __ballot_sync(0xffffffffu, slot >= 0 && slot % BS == BS - 1);
    const int h0 = blockIdx.y * kSummaryWarps, heads = min(kSummaryWarps, a.num_kv_heads - h0);
    const int items = __popc(ends) * heads;
    for (int it = warp; it < items; it += kSummaryWarps) {
        const int nth = it / heads, h = h0 + it - nth * heads;
        uint32_t rest = ends;
        for (int k = 0; k < nth; ++k) rest &= rest - 1;
        const int64_t blk = __shfl_sync(0xffffffffu, slot, __ffs(rest) - 1) / BS;
        const int64_t row = blk * a.num_kv_heads + h;
        const uint8_t *src = a.k_cache + row * (BS * D * ELEM) + lane * 16;
        uint4 w[LOADS];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) w[i] = *reinterpret_cast<const uint4 *>(src + i * 512);
        T hi[PAIRS], lo[PAIRS];  // E4M3: bytes 0 and 2 of a word, then 1 and 3
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int k = 0; k < PAIRS; ++k) {
                const uint32_t v = !FP8 ? u[k % 4] : (k & 1 ? u[k / 2] : u[k / 2 % 4] << 8) & 0xff00ff00u;
                const T x = pair(v);
                hi[k] = i == 0 ? x : __hmax2_nan(hi[k], x);
                lo[k] = i == 0 ? x : __hmin2_nan(lo[k], x);
            }
        }
        // lower half: the largest; upper half: the least
        T ext[PAIRS];
        float amax = 0.f;
        bool odd = false;
#pragma unroll
        for (int k = 0; k < PAIRS; ++k) {
            const bool low = lane < 16;
            T x = low ? hi[k] : lo[k];
#pragma unroll
            for (int m = 16; m >= LPR; m >>= 1) {
                const T o = pair(__shfl_xor_sync(0xffffffffu, m == 16 ? bits(low ? lo[k] : hi[k]) : bits(x), m));
                x = low ? __hmax2_nan(x, o) : __hmin2_nan(x, o);
            }
            ext[k] = x;
        }
        float2 val[PAIRS];
#pragma unroll
        for (int k = 0; k < PAIRS; ++k) {
            if constexpr (FP8) {
                const uint32_t b = bits(ext[k]);
                uint32_t f, none;
                e4m3x4_to_f16x2x2((b >> 8 & 0xffu) | (b >> 16 & 0xff00u), f, none);
                val[k] = __half22float2(*reinterpret_cast<const __half2 *>(&f));
            } else {
                val[k] = __bfloat1622float2(ext[k]);
            }
            odd |= !(fabsf(val[k].x) < INFINITY) || !(fabsf(val[k].y) < INFINITY);
            amax = fmaxf(amax, fmaxf(fabsf(val[k].x), fabsf(val[k].y)));
        }
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
        odd = __any_sync(0xffffffffu, odd);
        const int ex = odd ? kOddExp : shared_exponent(amax);
        const float inv = power_of_two(odd ? 0 : -ex);
        if ((lane & 15) < LPR) {
            uint32_t out[EPL / 4];
#pragma unroll
            for (int k = 0; k < EPL / 4; ++k) {
                // elements 4k .. 4k + 3
                const float2 p = val[2 * k], r = val[2 * k + 1];
                const int x[4] = {to_int8(p.x, inv), to_int8(FP8 ? r.x : p.y, inv), to_int8(FP8 ? p.y : r.x, inv),
                                  to_int8(r.y, inv)};
                uint32_t v = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b) v |= (static_cast<uint32_t>(x[b]) & 0xffu) << (8 * b);
                out[k] = odd ? 0u : v;
            }
            int8_t *dst = a.summary + row * (2 * D) + (lane < 16 ? 0 : D) + (lane & 15) * EPL;
            if constexpr (EPL == 16)
                *reinterpret_cast<uint4 *>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
            else
                *reinterpret_cast<uint2 *>(dst) = make_uint2(out[0], out[1]);
        }
        if (lane == 0) a.exponents[row] = static_cast<int8_t>(ex);
    }
}

// ---------------------------------------------------------------------------
// select
// ---------------------------------------------------------------------------

template <int D, int NT, int kSelThreads>
__global__ void __launch_bounds__(kSelThreads, (NT == 2 ? 384 : 512) / kSelThreads) select_kernel(const SelectArgs a) {
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ __align__(16) Choice<D, NT, kSelThreads> sh;
    dependent_wait();
    dependent_release();
    choose<D, NT, kSelThreads>(a, dyn, reinterpret_cast<uint32_t *>(dyn + copy_bytes(kSelThreads, D, a.stages)), sh,
                               static_cast<int>(cluster_rank()), static_cast<int>(cluster_size()), blockIdx.y, blockIdx.z);
}

template <int D, int NT, int kSelThreads>
static pa_status launch_threads(SelectArgs a, int num_rows, int ranks, cudaStream_t stream) {
    a.stages = kMaxStages;
    while (a.max_blocks > kMaxKeys * ranks) ranks *= 2;  // at most 8, by the limit on the table
    auto kern = select_kernel<D, NT, kSelThreads>;
    static std::atomic<uint64_t> raised{0};
    const int copies = copy_bytes(kSelThreads, D, kMaxStages);
    pa_status st = raise_smem_limit(reinterpret_cast<const void *>(kern), copies + key_bytes(kMaxKeys, 1), raised);
    if (st != PA_OK) return st;
    return cuda_check(launch_dependent(kern, dim3(ranks, a.num_kv_heads, num_rows), kSelThreads,
                                       copies + key_bytes(a.max_blocks, ranks), ranks, stream, a),
                      "sparse select launch");
}

// Up to a row to an SM: CTAs of 256 threads, several to a row while each has an SM
// to itself and enough pages to pay for the cluster's barriers (8 rows of 625 pages: 6.7
// us with eight, 8.0 with four; 16 of 2500: 11.4 with four, 12.4 with eight; of 313: 6.0
// with four, 8.0 with one; 72 of 625: 11.6 with two, 9.2 with one; of 2500: 19.3 and
// 25.1), or, of very many pages, of 128 threads, three to an SM (48 of 8192 pages: 27.8
// us with eight, 37.5 with two of 256; 96 of 2500: 19.8 with four, 24.8 with one of 256).
// Beyond, the fullest SM counts: 192 rows of 157 pages take 7.8 us with 128 threads and
// 8.8 with 256, of 625 15.5 and 13.5 (16.6 and 19.4 with 16 query heads, where one CTA of
// 256 fits an SM), of 2500 31.0 with two of 128 and 43.5 with one of 256; 1024 rows of
// 157 18.3 and 25.2.
template <int D, int NT>
static pa_status launch_select(const SelectArgs &a, int num_rows, cudaStream_t stream) {
    const int64_t rows = static_cast<int64_t>(num_rows) * a.num_kv_heads;
    const int pages = a.max_blocks;
    int threads = 256, ranks = 1;
    if (rows <= kSms) {
        if (rows * 16 <= kSms && pages > 256)
            ranks = 8;
        else if (rows * 4 <= kSms && pages > 128)
            ranks = 4;
        else if (rows * 8 <= 3 * kSms && pages >= 2000)
            threads = 128, ranks = 8;
        else if (rows * 2 <= kSms && pages >= 1000)
            ranks = 2;
        else if (rows * 2 > kSms && rows * 4 <= 3 * kSms && pages >= 2000)
            threads = 128, ranks = 4;
    } else {
        const bool two = rows * 2 <= 3 * kSms && pages >= 1000;  // the fullest SM has three
        if (rows > 2 * kSms || pages < 400 || NT == 2) threads = 128;
        if (two || pages >= 5000) threads = 128, ranks = 2;
    }
    return threads == 256 ? launch_threads<D, NT, 256>(a, num_rows, ranks, stream)
                          : launch_threads<D, NT, 128>(a, num_rows, ranks, stream);
}

pa_status check_select(int num_rows, int num_q_heads, int num_kv_heads, int head_dim, int num_blocks,
                       int block_size, int max_blocks, int top_k, int sink, int recent) {
    if (num_rows < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_blocks <= 0 || max_blocks <= 0)
        return fail(PA_ERR_INVALID_ARG,
                    "bad size (num_rows=%d, num_q_heads=%d, num_kv_heads=%d, num_blocks=%d, max_blocks_per_seq=%d)",
                    num_rows, num_q_heads, num_kv_heads, num_blocks, max_blocks);
    if (num_q_heads % num_kv_heads != 0)
        return fail(PA_ERR_INVALID_ARG, "num_q_heads %d is not a multiple of num_kv_heads %d",
                    num_q_heads, num_kv_heads);
    if (num_q_heads / num_kv_heads > 16)
        return fail(PA_ERR_UNSUPPORTED, "query group of %d heads (supported: 1..16)",
                    num_q_heads / num_kv_heads);
    if (head_dim != 64 && head_dim != 128)
        return fail(PA_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", head_dim);
    if (block_size != 16 && block_size != 32)
        return fail(PA_ERR_UNSUPPORTED, "block_size %d (supported: 16, 32)", block_size);
    if (static_cast<int64_t>(max_blocks) * block_size > 0x7fffffffLL)
        return fail(PA_ERR_INVALID_ARG, "max_blocks_per_seq * block_size exceeds 2^31");
    if (static_cast<int64_t>(num_blocks) * num_kv_heads * block_size > 0x7fffffffLL)
        return fail(PA_ERR_UNSUPPORTED, "pool of %d blocks x %d heads x %d rows exceeds 2^31 rows",
                    num_blocks, num_kv_heads, block_size);
    if (num_rows > 65535 || num_kv_heads > 65535)
        return fail(PA_ERR_UNSUPPORTED, "more than 65535 rows or KV heads");
    if (top_k <= 0 || sink < 0 || recent < 1)
        return fail(PA_ERR_INVALID_ARG, "bad choice (top_k=%d, sink_blocks=%d, recent_blocks=%d): the page being "
                    "filled is always read, so recent_blocks is 1 or more", top_k, sink, recent);
    if (static_cast<int64_t>(sink) + recent > top_k)
        return fail(PA_ERR_INVALID_ARG, "sink_blocks %d + recent_blocks %d exceed top_k %d", sink, recent, top_k);
    if (top_k > kMaxTableBlocks)
        return fail(PA_ERR_UNSUPPORTED, "top_k %d (supported: up to %d)", top_k, kMaxTableBlocks);
    if (max_blocks > kMaxTableBlocks)
        return fail(PA_ERR_UNSUPPORTED, "max_blocks_per_seq %d (supported: up to %d)", max_blocks, kMaxTableBlocks);
    return PA_OK;
}

SelectArgs select_args(const void *q, const int8_t *summary, const int8_t *exponents, const int32_t *block_tables,
                       int max_blocks, const int32_t *context_lens, int num_q_heads, int num_kv_heads, int num_blocks,
                       int block_size, int top_k, int sink, int recent, int32_t *selected, int32_t *counts) {
    SelectArgs a;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.summary = summary;
    a.exponents = exponents;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.selected = selected;
    a.counts = counts;
    a.max_blocks = max_blocks;
    a.num_blocks = num_blocks;
    a.num_kv_heads = num_kv_heads;
    a.group = num_q_heads / num_kv_heads;
    a.block_size = block_size;
    a.top_k = top_k;
    a.sink = sink;
    a.recent = recent;
    a.err = device_error_word();
    return a;
}

pa_status run_select(const SelectArgs &a, int num_rows, int head_dim, cudaStream_t stream) {
    if (!a.err) return fail(PA_ERR_CUDA, "cannot resolve the device error word");
    if (head_dim == 128)
        return a.group <= 8 ? launch_select<128, 1>(a, num_rows, stream) : launch_select<128, 2>(a, num_rows, stream);
    return a.group <= 8 ? launch_select<64, 1>(a, num_rows, stream) : launch_select<64, 2>(a, num_rows, stream);
}

template <int D, int BS>
static cudaError_t launch_summary(const SummaryArgs &a, bool fp8, dim3 grid, cudaStream_t stream) {
    return fp8 ? launch_dependent(summary_kernel<D, BS, true>, grid, kSummaryWarps * 32, 0, 0, stream, a)
               : launch_dependent(summary_kernel<D, BS, false>, grid, kSummaryWarps * 32, 0, 0, stream, a);
}

}  // namespace sparse
}  // namespace pa

using namespace pa;
using namespace pa::sparse;

extern "C" {

pa_status pa_block_summary(const void *k_cache, const int32_t *slot_mapping, int num_tokens,
                           int num_blocks, int num_kv_heads, int head_dim, int block_size,
                           pa_kv_dtype kv_dtype, int8_t *summary, int8_t *exponents,
                           cudaStream_t stream) {
    clear_error();
    if (num_tokens < 0 || num_blocks <= 0 || num_kv_heads <= 0)
        return fail(PA_ERR_INVALID_ARG, "bad size (num_tokens=%d, num_blocks=%d, num_kv_heads=%d)",
                    num_tokens, num_blocks, num_kv_heads);
    if (num_kv_heads > 65535) return fail(PA_ERR_UNSUPPORTED, "more than 65535 KV heads");
    if (head_dim != 64 && head_dim != 128)
        return fail(PA_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", head_dim);
    if (block_size != 16 && block_size != 32)
        return fail(PA_ERR_UNSUPPORTED, "block_size %d (supported: 16, 32)", block_size);
    if (kv_dtype != PA_KV_BF16 && kv_dtype != PA_KV_FP8_E4M3)
        return fail(PA_ERR_UNSUPPORTED, "kv_dtype %d", static_cast<int>(kv_dtype));
    if (static_cast<int64_t>(num_blocks) * block_size > 0x7fffffffLL)
        return fail(PA_ERR_UNSUPPORTED, "pool of %d blocks exceeds 2^31 slots", num_blocks);
    if (num_tokens == 0) return PA_OK;
    if (!k_cache || !slot_mapping || !summary || !exponents) return fail(PA_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(k_cache) || !aligned16(summary))
        return fail(PA_ERR_INVALID_ARG, "k_cache and summary must be 16-byte aligned");
    unsigned int *err = device_error_word();
    if (!err) return fail(PA_ERR_CUDA, "cannot resolve the device error word");
    SummaryArgs a;
    a.k_cache = static_cast<const uint8_t *>(k_cache);
    a.slots = slot_mapping;
    a.summary = summary;
    a.exponents = exponents;
    a.num_slots = static_cast<int64_t>(num_blocks) * block_size;
    a.num_tokens = num_tokens;
    a.num_kv_heads = num_kv_heads;
    a.err = err;
    const bool fp8 = kv_dtype == PA_KV_FP8_E4M3;
    // Few tokens may all complete a page (sequences of one length), many are mostly
    // runs of a sequence: a CTA takes one slot up to some 500, 16 from 4096 on (8 heads,
    // 256 sequences that all complete a page: 2.9 us, 16.8 with 16 slots to a CTA; runs
    // of 4096 tokens in all: 2.9 us with 16, 3.7 with 6).
    a.per_cta = std::max(1, std::min(kSummarySlots, num_tokens / 256));
    const dim3 grid((static_cast<unsigned>(num_tokens) + a.per_cta - 1) / a.per_cta,
                    (num_kv_heads + kSummaryWarps - 1) / kSummaryWarps);
    const cudaError_t e = head_dim == 128 ? (block_size == 16 ? launch_summary<128, 16>(a, fp8, grid, stream)
                                                              : launch_summary<128, 32>(a, fp8, grid, stream))
                                          : (block_size == 16 ? launch_summary<64, 16>(a, fp8, grid, stream)
                                                              : launch_summary<64, 32>(a, fp8, grid, stream));
    return cuda_check(e, "block summary launch");
}

pa_status pa_sparse_select(const void *q, const int8_t *summary, const int8_t *exponents,
                           const int32_t *block_tables, int max_blocks_per_seq,
                           const int32_t *context_lens, int num_rows, int num_q_heads,
                           int num_kv_heads, int head_dim, int num_blocks, int block_size, int top_k,
                           int sink_blocks, int recent_blocks, int32_t *selected, int32_t *counts,
                           cudaStream_t stream) {
    clear_error();
    pa_status st = check_select(num_rows, num_q_heads, num_kv_heads, head_dim, num_blocks, block_size,
                                max_blocks_per_seq, top_k, sink_blocks, recent_blocks);
    if (st != PA_OK) return st;
    if (num_rows == 0) return PA_OK;
    if (!q || !summary || !exponents || !block_tables || !context_lens || !selected || !counts)
        return fail(PA_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(q) || !aligned16(summary))
        return fail(PA_ERR_INVALID_ARG, "q and summary must be 16-byte aligned");
    return run_select(select_args(q, summary, exponents, block_tables, max_blocks_per_seq, context_lens, num_q_heads,
                                  num_kv_heads, num_blocks, block_size, top_k, sink_blocks, recent_blocks, selected,
                                  counts),
                      num_rows, head_dim, stream);
}

}  // extern "C"
