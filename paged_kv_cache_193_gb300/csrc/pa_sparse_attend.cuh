// Decode attention over chosen pages: for each (row, KV head) the softmax of
// softmax_scale * q . K[t] over the tokens of the listed logical pages, applied
// to V ("vLLM PagedAttention: Memory Optimization & High-Throughput LLM
// Inference Tuning", section 2, walks every page; here only those of a list
// are walked).
//
// One cluster of CTAs per (row, KV head), the list dealt out over the
// cluster's warps.  A warp keeps several pages in flight: TMA tile loads of
// the K and V page into a ring stage of its own, S^T = K Q^T as m16n8k16
// products with the query group (padded to 8 or 16) as N, one pass of online
// softmax, O^T += V^T P^T.  The CTA's warps, then the cluster's CTAs over
// distributed shared memory, join their (max, sum, accumulator) triples, so
// there is no workspace and no second kernel however few rows there are.
//
// Bound by memory: a page is read once and used for all queries of its KV head.
// 64 sequences of 4K-32K tokens, 64 / 8 heads, top 128: 689 MB in 113 us with the
// choice, 6.1 TB/s (0.90 of a copy's rate); 256 sequences of 512-2,048 tokens, top
// 32: 575 MB in 100.6 us, 5.7 TB/s.  Over a list that is there the pages alone take
// 80 us in both, 6.7 TB/s.  With few rows by latency: one sequence of 5,003 tokens,
// top 64, 10.4 us.
//
// The same kernel attends to what a sequence has behind a prefix that it shares
// (SUFFIX): the list is the pages from there on, and the parts that the prefix's
// kernel left (pa_rows.cuh) join the warps' own at the end.
#pragma once

#include <cudaTypedefs.h>

#include <algorithm>
#include <type_traits>

#include "pa_rows.cuh"
#include "pa_sparse_select.cuh"

namespace pa {
namespace sparse {

// What attends to a whole sequence when part of it has been attended to before.
struct Prefix {
    const int32_t *group_start;    // [num_groups + 1] first sequence of each group
    const int32_t *prefix_blocks;  // [num_groups]
    int num_groups, max_blocks;    // no prefix counts for more pages than this
    int parts;                     // of each prefix; 0: there are none
    const float *o;                // [parts][rows][head_dim]
    const float2 *ml;              // [parts][rows]
    int64_t rows;
    // Null: the rest's kernel makes the join, and waits for the prefix's.  Else it leaves
    // a part of its own, [rows][head_dim] and [rows], for another kernel to join.
    float *rest_o;
    float2 *rest_ml;
};

struct Args {
    const __nv_bfloat16 *q;
    const int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *selected;  // [num_rows][num_kv_heads][top_k] logical pages
    const int32_t *counts;    // [num_rows][num_kv_heads]
    __nv_bfloat16 *out;
    int max_blocks, num_blocks, num_q_heads, num_kv_heads, group, top_k;
    float softmax_log2;  // softmax_scale * log2(e): scores in base-2 units
    float kv_scale;
    const float *k_scales, *v_scales;
    unsigned int *err;
    uint64_t wait_limit_ns;
    int stall_first_wait;
    SelectArgs select;  // of the kernel that chooses the pages itself
    int longest_first;  // its clusters take the rows by length
    Prefix prefix;      // of the kernel that attends behind a prefix
    // of several tokens' rows (kRows): sequence s's are query_start[s] .. query_start[s + 1] - 1
    const int32_t *query_start;
    int num_tokens, max_query_len;
};

// A list of pages, pages that the kernel chooses, the pages behind a prefix
// (kSuffix; kSuffixHeads: a warp to a KV head), or all pages, for up to 16 rows
// (tokens times query heads of a KV head).
enum Mode { kList, kChoose, kSuffix, kSuffixHeads, kRows };

pa_status launch_chosen(int head_dim, int block_size, bool fp8, const CUtensorMap &tk, const CUtensorMap &tv, const Args &a,
                        int num_rows, int splits, int warps, cudaStream_t stream);

// CTAs of four warps to an SM, as the registers and the ring allow; half as
// many of eight warps.
constexpr int resident_ctas(int head_dim, int block_size, bool fp8, int group) {
    const bool big = block_size == 32 && !fp8;  // pages twice the others' size
    if (group <= 8) return big ? 3 : 4;
    return head_dim == 64 || (block_size == 16 && !fp8) ? 3 : 2;
}

// limit of the drain of copies in flight after a wait gave up
constexpr uint64_t kDrainNs = 2000000000ull;

template <int D, int BS, bool FP8, int NT, int NW, int SPW>
struct Shape {
    static constexpr int ELEM = FP8 ? 1 : 2;
    static constexpr int ROWB = D * ELEM;                  // bytes of a token's row
    static constexpr int SLAB = ROWB >= 128 ? 128 : ROWB;  // TMA box width = swizzle span
    static constexpr int NSLAB = ROWB / SLAB;
    static constexpr int PAGE = BS * ROWB;
    static constexpr int PPI = (FP8 && BS == 16) ? 2 : 1;  // pages per step of a warp
    static constexpr int STAGE = 2 * PPI * PAGE;           // K pages, then V pages
    static constexpr int NSTAGE = NW * SPW;
    static constexpr int RING = NSTAGE * STAGE;
    static constexpr int NP = 8 * NT;  // group padded to the product's N
    static constexpr int OSTR = D + 4;
    // the join: a partial output per warp, (reference, sum) per warp and head,
    // then the CTA's own partial and (reference, sum)
    static constexpr int JOIN = (NW * NP * OSTR + 2 * NW * NP + NP * D + 2 * NP) * 4;
    static constexpr int SMEM = (RING > JOIN ? RING : JOIN) + 1024;  // + base alignment
    static constexpr int MT = BS / 16;   // 16-token tiles of a page
    static constexpr int MI = PPI * MT;  // and of a step
    static constexpr int KSTEPS = D / 16;
    static constexpr int DT = D / 16;
    static constexpr int CPT = D / 64;  // E4M3: 16-byte pieces per thread and row
    static constexpr int TERMS = FP8 ? 1 : 2;  // numbers that a probability goes into P V as
};

// The upper of the two bf16 numbers that stand for a probability; `p` becomes the
// lower, still to be rounded: together they are off by less than 2^-14 of it, and
// what is left of the output's error is its own rounding (64 sequences of 4K-32K
// tokens: 0.0017 of its norm, as with sums in 32 bits throughout; 0.0025 with one
// bf16 number, which takes 1% less time, 113.8 and 114.9 us).  The upper is a little
// less than p cut off, so the lower is positive like it, whatever p > 0: an
// infinite value times the two stays infinite, where a rest of 0 or below would
// make it a NaN.
__device__ __forceinline__ float split_bf16(float &p) {
    const float upper = __uint_as_float(__float_as_uint(p * 0.998046875f) & 0xffff0000u);  // 1 - 2^-9
    p -= upper;
    return upper;
}

// Address of byte b of token row t in a page tile as the TMA's swizzle lays
// it down.
template <class C, int BS>
__device__ __forceinline__ uint32_t at(uint32_t base, int t, int b) {
    const int slab = b / C::SLAB, within = b % C::SLAB, chunk = within >> 4;
    const int phys = C::SLAB == 128 ? (chunk ^ (t & 7)) : (chunk ^ ((t >> 1) & 3));
    return base + slab * (BS * C::SLAB) + t * C::SLAB + (phys << 4) + (within & 15);
}

// The row of the z-th longest context of `n` (at most kMaxSorted), the first of
// equals first; `room` is 4 n + 4 bytes of shared memory.
constexpr int kMaxSorted = 128;
__device__ __forceinline__ int longest_row(const int32_t *lens, int n, int z, void *room) {
    int32_t *len = static_cast<int32_t *>(room);
    const int i = threadIdx.x;
    const int32_t mine = i < n ? __ldcg(lens + i) : 0;
    if (i < n) len[i] = mine;
    __syncthreads();
    int before = 0;
    for (int j = 0; j < n; ++j) before += len[j] > mine || (len[j] == mine && j < i);
    if (i < n && before == z) len[n] = i;
    __syncthreads();
    const int row = len[n];
    // The room is used again, by page copies too: a barrier alone does not order these
    // accesses before what the copies write.
    fence_proxy_async_smem();
    __syncthreads();
    return row;
}

// Pages that sequence s, of n tokens, shares with its group: 0, or all of the
// group's prefix.  Called by whole warps.  The loads pass by the first-level cache:
// this runs before the kernel in front has ended.
__device__ __forceinline__ int shared_pages(const Prefix &p, int s, int n, int block_size) {
    if (p.parts == 0 || p.num_groups == 0) return 0;
    const int lane = threadIdx.x & 31;
    int lo = 0, size = p.num_groups;
    // the last group that starts at s or before, among 32 and then 32 of those between
    while (size > 32) {
        const int step = (size + 31) / 32, at = lane * step;
        const int v = at < size ? __ldcg(p.group_start + lo + at) : 0x7fffffff;
        const int count = __popc(__ballot_sync(0xffffffffu, v <= s));
        if (count == 0) return 0;
        const int skip = min((count - 1) * step, size - 1);
        lo += skip;
        size = min(step, size - skip);
    }
    // at last all that may be wanted is on its way at once
    const bool has = lane < size;
    const int begin = has ? __ldcg(p.group_start + lo + lane) : 0x7fffffff, end = has ? __ldcg(p.group_start + lo + lane + 1) : 0;
    const int blocks = has ? min(__ldcg(p.prefix_blocks + lo + lane), p.max_blocks) : 0;
    const int count = __popc(__ballot_sync(0xffffffffu, begin <= s));
    if (count == 0) return 0;
    const int pages = __shfl_sync(0xffffffffu, blocks, count - 1);
    return s < __shfl_sync(0xffffffffu, end, count - 1) && pages > 0 && n / block_size >= pages ? pages : 0;
}

__device__ __forceinline__ bool grids_last() {
    return blockIdx.x + 1 == gridDim.x && blockIdx.y + 1 == gridDim.y && blockIdx.z + 1 == gridDim.z;
}

// kChoose: the cluster first chooses the row's pages, in the ring's memory.
// kSuffix: launched when the prefix's kernel is on the SMs, which has waited for
// those before it; only the join waits for that kernel.
template <int D, int BS, bool FP8, int NT, int NW, int SPW, int MODE>
__global__ void __launch_bounds__(NW * 32, resident_ctas(D, BS, FP8, NT * 8) * 4 / NW)
    attend_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const Args a) {
    using C = Shape<D, BS, FP8, NT, NW, SPW>;
    constexpr int PPI = C::PPI, MI = C::MI;
    constexpr bool CHOOSE = MODE == kChoose, HEADS = MODE == kSuffixHeads, SUFFIX = MODE == kSuffix || HEADS, ROWS = MODE == kRows;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[C::NSTAGE];
    __shared__ __align__(8) uint64_t stall_bar;  // never completed (wait-limit test hook)

    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t ring = (raw + 1023u) & ~1023u;
    float *join = reinterpret_cast<float *>(smem_raw + (ring - raw));
    const uint32_t rank = cluster_rank(), ranks = cluster_size();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = lane >> 2, c = lane & 3;
    const bool idle = HEADS && static_cast<int>(blockIdx.y) * NW + warp >= a.num_kv_heads;  // a warp without a head
    const int h = !HEADS ? blockIdx.y : idle ? 0 : blockIdx.y * NW + warp;
    int s = blockIdx.z;

    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < C::NSTAGE; ++i) mbar_init(smem_addr(&bars[i]), 1);
        mbar_init(smem_addr(&stall_bar), 1);
        fence_barrier_init();
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (!SUFFIX || a.prefix.parts == 0) dependent_wait();
    if constexpr (CHOOSE || SUFFIX)
        if (a.longest_first) s = longest_row(a.context_lens, gridDim.z, s, join);

    // plain loads; past the first-level cache where the kernel in front still runs
    auto load = [](const auto *p) { return SUFFIX ? __ldcg(p) : *p; };
    const float k_scale = FP8 ? (a.k_scales ? load(a.k_scales + h) : a.kv_scale) : 1.f;
    const float v_scale = FP8 ? (a.v_scales ? load(a.v_scales + h) : a.kv_scale) : 1.f;
    const float score_scale = a.softmax_log2 * k_scale;

    Chosen chosen{0, nullptr};
    if constexpr (CHOOSE) {
        __shared__ __align__(16) Choice<D, NT, NW * 32> sh;
        uint8_t *mem = smem_raw + (ring - raw);
        chosen = choose<D, NT, NW * 32>(a.select, mem, reinterpret_cast<uint32_t *>(mem + copy_bytes(NW * 32, D, a.select.stages)), sh,
                                        static_cast<int>(rank), static_cast<int>(ranks), h, s);
        fence_proxy_async_smem();  // this memory is next written by page copies
    }

    // Rows of queries, and where each begins: the group's heads, or those of several tokens.
    int num_live = a.group, token0 = s;
    if constexpr (ROWS) {
        const int end = a.query_start[s + 1];
        token0 = a.query_start[s];
        if (token0 < 0 || end < token0 || end > a.num_tokens || end - token0 > a.max_query_len) {
            if (tid == 0 && rank == 0) set_device_error(a.err, PA_DEVERR_BAD_CONTEXT);
            num_live = 0;
        } else {
            num_live = (end - token0) * a.group;
        }
    }
    auto row_at = [&](int g) -> int64_t {
        if constexpr (ROWS) {
            const int t = g / a.group;
            return ((static_cast<int64_t>(token0) + t) * a.num_q_heads + h * a.group + (g - t * a.group)) * D;
        } else {
            return (static_cast<int64_t>(token0) * a.num_q_heads + h * a.group + g) * D;
        }
    };

    // query fragments (B operand of S^T = K Q^T), resident in registers
    uint32_t qf[C::KSTEPS][NT][2];
    {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int g = nt * 8 + r;
            const bool live = g < num_live;
            const __nv_bfloat16 *qg = a.q + row_at(live ? g : 0);
#pragma unroll
            for (int kk = 0; kk < C::KSTEPS; ++kk) {
                if constexpr (!FP8) {
                    qf[kk][nt][0] = live ? load(reinterpret_cast<const uint32_t *>(qg + kk * 16 + 2 * c)) : 0u;
                    qf[kk][nt][1] = live ? load(reinterpret_cast<const uint32_t *>(qg + kk * 16 + 8 + 2 * c)) : 0u;
                } else {
                    // permuted order, as the K bytes below: this thread's dims
                    // are c*16*CPT + 4*kk + {0,1,2,3}
                    const uint2 w = live ? load(reinterpret_cast<const uint2 *>(qg + c * 16 * C::CPT + 4 * kk))
                                         : make_uint2(0u, 0u);
                    const float2 f0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w.x));
                    const float2 f1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w.y));
                    qf[kk][nt][0] = pack2<true>(f0.x, f0.y);
                    qf[kk][nt][1] = pack2<true>(f1.x, f1.y);
                }
            }
        }
    }
    int n = load(a.context_lens + s);
    if (n > a.max_blocks * BS) {
        if (tid == 0 && rank == 0 && h == 0) set_device_error(a.err, PA_DEVERR_BAD_CONTEXT);
        n = a.max_blocks * BS;
    }
    const int nb = n > 0 ? (n + BS - 1) / BS : 0;
    __syncthreads();
    int skip = 0;  // pages in front of the list's first
    if constexpr (SUFFIX) {
        skip = shared_pages(a.prefix, s, n, BS);
        chosen = Chosen{idle ? 0 : nb - skip, nullptr};
    } else if constexpr (ROWS) {
        chosen = Chosen{num_live ? nb : 0, nullptr};
    } else if constexpr (!CHOOSE) {
        const int64_t row = static_cast<int64_t>(s) * a.num_kv_heads + h;
        chosen = Chosen{min(max(a.counts[row], 0), a.top_k), a.selected + row * a.top_k};
    }

    // ---- this warp's entries of the list ----------------------------------------
    const int step = HEADS ? 1 : NW * static_cast<int>(ranks);
    const int first = HEADS ? 0 : static_cast<int>(rank) * NW + warp;
    // logical page of the warp's k-th entry
    auto entry = [&](int k) -> int {
        const int i = first + k * step;
        return SUFFIX ? skip + i : ROWS ? i : chosen.list ? chosen.list[i] : i;
    };
    const int32_t *table = a.block_tables + static_cast<int64_t>(s) * a.max_blocks;
    const int my_pages = chosen.count > first ? (chosen.count - first + step - 1) / step : 0;
    const int my_steps = (my_pages + PPI - 1) / PPI;
    const uint64_t policy = l2_evict_first_policy();
    const int rows_total = a.num_blocks * a.num_kv_heads * BS;

    // First tensor row of the warp's k-th page; rows_total (outside: the copy
    // fills zeros) for an entry that is no page of the sequence or pool.
    auto first_row = [&](int k) -> int {
        if (k >= my_pages) return rows_total;
        const int j = entry(k);
        if (j < 0 || j >= nb) {
            set_device_error(a.err, PA_DEVERR_BAD_BLOCK);
            return rows_total;
        }
        const int b = load(table + j);
        if (b < 0 || b >= a.num_blocks) {
            set_device_error(a.err, PA_DEVERR_BAD_BLOCK);
            return rows_total;
        }
        return (b * a.num_kv_heads + h) * BS;
    };
    int y_cur = first_row(lane), y_next = first_row(32 + lane), chunk = 0;
    auto page_row = [&](int k) -> int {  // called by all lanes with k = 0, 1, 2, ...
        if ((k >> 5) != chunk) {
            y_cur = y_next;
            chunk = k >> 5;
            y_next = first_row((chunk + 1) * 32 + lane);
        }
        return __shfl_sync(0xffffffffu, y_cur, k & 31);
    };
    auto fetch = [&](int it) {
        int ys[PPI];
#pragma unroll
        for (int p = 0; p < PPI; ++p) ys[p] = page_row(PPI * it + p);
        const int live = min(PPI, my_pages - PPI * it);
        if (lane >= live) return;
        const int st = warp * SPW + it % SPW;
        const uint32_t bar = smem_addr(&bars[st]);
        if (lane == 0) mbar_arrive_expect_tx(bar, live * 2 * C::PAGE);
        const uint32_t kdst = ring + st * C::STAGE + lane * C::PAGE;
        const uint32_t vdst = kdst + PPI * C::PAGE;
        int y = ys[0];
#pragma unroll
        for (int p = 1; p < PPI; ++p)
            if (lane == p) y = ys[p];
#pragma unroll
        for (int sl = 0; sl < C::NSLAB; ++sl) {
            tma_load_2d(kdst + sl * (BS * C::SLAB), &tmK, sl * (C::SLAB / C::ELEM), y, bar, policy);
            tma_load_2d(vdst + sl * (BS * C::SLAB), &tmV, sl * (C::SLAB / C::ELEM), y, bar, policy);
        }
    };
    const int prolog = my_steps < SPW ? my_steps : SPW;
    for (int it = 0; it < prolog; ++it) fetch(it);

    float o[C::DT][NT][4];
#pragma unroll
    for (int dt = 0; dt < C::DT; ++dt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[dt][nt][e] = 0.f;
    // probabilities are taken against m_ref, which moves only when a tile's
    // maximum exceeds it by more than kLazy (base-2 units): they stay below
    // 2^kLazy and the accumulator is rescaled rarely
    constexpr float kLazy = 8.f;
    // With an E4M3 cache they go into P V in fp16, which holds V's codes: rounded by
    // 2^-11, an eighth of the output's own rounding, down to 2^-14 and ever more
    // below.  Taken times 2^7 they stay in its range, up to 2^15, and keep their bits
    // down to 2^-21 (a long list's small ones add up: outputs of 6000 tokens, most at
    // 2^-23, were up to 14% off without).
    constexpr float kRaise = 7.f;
    float m_ref[NT][2], l_run[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            m_ref[nt][j] = -INFINITY;
            l_run[nt][j] = 0.f;
        }
    // Token (within its 16-token tile) of MMA row r, and of row r + 8: the
    // E4M3 V fragments pair tokens 4c, 4c+1 and 4c+2, 4c+3, and the scores
    // take the same order.
    const int tok_r = FP8 ? (r >> 1) * 4 + (r & 1) : r;
    const int tok_dh = FP8 ? 2 : 8;

    bool ok = true;
    int it_fail = 0;
    if (a.stall_first_wait && my_steps > 0)
        ok = mbar_wait_bounded(smem_addr(&stall_bar), 0, a.wait_limit_ns);
    for (int it = 0; ok && it < my_steps; ++it) {
        const int st = warp * SPW + it % SPW;
        // tokens of the step's pages (a list entry read again: it is cached)
        int valid[PPI];
        bool any = false;
#pragma unroll
        for (int p = 0; p < PPI; ++p) {
            const int k = PPI * it + p;
            const int j = k < my_pages ? entry(k) : -1;
            valid[p] = j >= 0 && j < nb ? min(BS, n - j * BS) : 0;
            any |= valid[p] > 0;
        }
        if (!mbar_wait_bounded(smem_addr(&bars[st]), (it / SPW) & 1, a.wait_limit_ns)) {
            ok = false;
            it_fail = it;
            break;
        }
        const uint32_t kbase = ring + st * C::STAGE;
        const uint32_t vbase = kbase + PPI * C::PAGE;
        if (any) {
            bool partial = false;
#pragma unroll
            for (int p = 0; p < PPI; ++p) partial |= valid[p] < BS;
            if (partial) {
                // rows behind the context hold anything: zero V so that a
                // probability of 0 times them is 0
                constexpr int CH = C::NSLAB * (C::SLAB / 16);
#pragma unroll
                for (int p = 0; p < PPI; ++p) {
                    const uint32_t vb = vbase + p * C::PAGE;
                    for (int i = lane; i < (BS - valid[p]) * CH; i += 32) {
                        const int row = valid[p] + i / CH, rem = i % CH;
                        sts128_zero(vb + (rem / (C::SLAB / 16)) * (BS * C::SLAB) + row * C::SLAB +
                                    (rem % (C::SLAB / 16)) * 16);
                    }
                }
                fence_proxy_async_smem();  // before the stage's next copy
                __syncwarp();
            }

            float sc[MI][NT][4];
#pragma unroll
            for (int mi = 0; mi < MI; ++mi)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[mi][nt][e] = 0.f;
            if constexpr (!FP8) {
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) {
                    const uint32_t kb = kbase + (mi / C::MT) * C::PAGE;
                    const int t = (mi % C::MT) * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
                    for (int kk = 0; kk < C::KSTEPS; ++kk) {
                        uint32_t a0, a1, a2, a3;
                        ldsm_x4(at<C, BS>(kb, t, (kk * 16 + (lane >> 4) * 8) * 2), a0, a1, a2, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816<false>(sc[mi][nt], a0, a1, a2, a3, qf[kk][nt][0], qf[kk][nt][1]);
                    }
                }
            } else {
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) {
                    const uint32_t kb = kbase + (mi / C::MT) * C::PAGE;
                    const int t0 = (mi % C::MT) * 16 + tok_r, t1 = t0 + tok_dh;
                    uint4 ra[C::CPT], rb[C::CPT];
#pragma unroll
                    for (int j = 0; j < C::CPT; ++j) {
                        ra[j] = lds128(at<C, BS>(kb, t0, (c * C::CPT + j) * 16));
                        rb[j] = lds128(at<C, BS>(kb, t1, (c * C::CPT + j) * 16));
                    }
#pragma unroll
                    for (int kk = 0; kk < C::KSTEPS; ++kk) {
                        const uint4 &A = ra[kk / 4];
                        const uint4 &B = rb[kk / 4];
                        const uint32_t wa = (kk % 4 == 0) ? A.x : (kk % 4 == 1) ? A.y : (kk % 4 == 2) ? A.z : A.w;
                        const uint32_t wb = (kk % 4 == 0) ? B.x : (kk % 4 == 1) ? B.y : (kk % 4 == 2) ? B.z : B.w;
                        uint32_t a0, a1, a2, a3;
                        e4m3x4_to_f16x2x2(wa, a0, a2);
                        e4m3x4_to_f16x2x2(wb, a1, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816<true>(sc[mi][nt], a0, a1, a2, a3, qf[kk][nt][0], qf[kk][nt][1]);
                    }
                }
            }

            // online softmax over the step's tokens, per query head
            float mx[NT][2];
            bool grow = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float m = -INFINITY;
#pragma unroll
                    for (int mi = 0; mi < MI; ++mi) {
                        const int lim = valid[mi / C::MT] - (mi % C::MT) * 16;
#pragma unroll
                        for (int hi = 0; hi < 2; ++hi) {
                            float x = sc[mi][nt][hi * 2 + j] * score_scale;
                            x = tok_r + hi * tok_dh < lim ? x : -INFINITY;
                            sc[mi][nt][hi * 2 + j] = x;
                            m = fmaxf(m, x);
                        }
                    }
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                    mx[nt][j] = m;
                    grow |= m - m_ref[nt][j] > kLazy;  // the difference: a large score's sum would round
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float m_new = fmaxf(m_ref[nt][j], mx[nt][j]);
                        const float alpha = m_new == -INFINITY ? 1.f : fast_exp2(m_ref[nt][j] - m_new);
                        m_ref[nt][j] = m_new;
                        l_run[nt][j] *= alpha;
#pragma unroll
                        for (int dt = 0; dt < C::DT; ++dt) {
                            o[dt][nt][j] *= alpha;
                            o[dt][nt][j + 2] *= alpha;
                        }
                    }
            }
            uint32_t pb[MI][NT][C::TERMS][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    // no finite score so far: any reference will do for the zeros
                    const float ref = m_ref[nt][j] == -INFINITY ? 0.f : m_ref[nt][j];
                    float sum = 0.f;
#pragma unroll
                    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
                        for (int hi = 0; hi < 2; ++hi) {
                            float y = sc[mi][nt][hi * 2 + j] - ref;
                            if constexpr (FP8) y += kRaise;  // not to the reference, which may be large
                            const float pr = fast_exp2(y);
                            sc[mi][nt][hi * 2 + j] = pr;
                            sum += pr;
                        }
                    l_run[nt][j] += sum;
                }
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) {
                    float(&p)[4] = sc[mi][nt];
                    if constexpr (!FP8) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float x = split_bf16(p[2 * i]), y = split_bf16(p[2 * i + 1]);
                            pb[mi][nt][1][i] =
                                movmatrix_trans(__byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632));
                        }
                    }
                    pb[mi][nt][0][0] = movmatrix_trans(pack2<FP8>(p[0], p[1]));
                    pb[mi][nt][0][1] = movmatrix_trans(pack2<FP8>(p[2], p[3]));
                }
            }

            // O^T += V^T P^T
            if constexpr (!FP8) {
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) {
                    const uint32_t vb = vbase + (mi / C::MT) * C::PAGE;
                    const int t = (mi % C::MT) * 16 + (lane & 7) + (lane >> 4) * 8;
#pragma unroll
                    for (int dt = 0; dt < C::DT; ++dt) {
                        uint32_t a0, a1, a2, a3;
                        ldsm_x4_trans(at<C, BS>(vb, t, (dt * 16 + ((lane >> 3) & 1) * 8) * 2), a0, a1, a2, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < C::TERMS; ++i)
                                mma16816<false>(o[dt][nt], a0, a1, a2, a3, pb[mi][nt][i][0], pb[mi][nt][i][1]);
                    }
                }
            } else {
#pragma unroll
                for (int mi = 0; mi < MI; ++mi) {
                    const uint32_t vb = vbase + (mi / C::MT) * C::PAGE;
                    const int t = (mi % C::MT) * 16 + (lane & 15);
#pragma unroll
                    for (int cp = 0; cp < D / 32; ++cp) {
                        uint32_t w0, w1, w2, w3, a0, a1, a2, a3;
                        ldsm_x2_trans_b8(at<C, BS>(vb, t, (2 * cp + (lane >> 4)) * 16), w0, w1, w2, w3);
                        e4m3x4_to_f16x2x2(w0, a0, a2);
                        e4m3x4_to_f16x2x2(w1, a1, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816<true>(o[2 * cp][nt], a0, a1, a2, a3, pb[mi][nt][0][0], pb[mi][nt][0][1]);
                        e4m3x4_to_f16x2x2(w2, a0, a2);
                        e4m3x4_to_f16x2x2(w3, a1, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816<true>(o[2 * cp + 1][nt], a0, a1, a2, a3, pb[mi][nt][0][0], pb[mi][nt][0][1]);
                    }
                }
            }
        }
        __syncwarp();
        if (it + SPW < my_steps) fetch(it + SPW);
    }
    if (!ok) {
        // a copy never arrived: flag it, wait (bounded) for the copies still in
        // flight into this warp's stages, and go on with nothing
        if (lane == 0) set_device_error(a.err, PA_DEVERR_TIMEOUT);
        const int issued = min(my_steps, it_fail + SPW);
        for (int it = it_fail; it < issued; ++it)
            mbar_wait_bounded(smem_addr(&bars[warp * SPW + it % SPW]), (it / SPW) & 1, kDrainNs);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m_ref[nt][0] = m_ref[nt][1] = -INFINITY;
            l_run[nt][0] = l_run[nt][1] = 0.f;
        }
    }

    // Not earlier: the next kernel's CTAs would take the places of this one's
    // (64 sequences of 4K-32K tokens: 114.7 us a pass with it at the start, 113.4
    // here; in E4M3 62.1 and 61.0).
    dependent_release();

    // ---- join the warps ---------------------------------------------------------
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float l = l_run[nt][j];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            l_run[nt][j] = l;
        }
    if constexpr (HEADS) {
        // A warp has a head to itself: its part joins the prefix's and leaves, through its
        // own share of the ring.
        static_assert(C::NP * (C::OSTR + rows::kMaxParts) * 4 <= SPW * C::STAGE, "a warp's output in its share of the ring");
        const bool apart = a.prefix.rest_o != nullptr;
        if (a.prefix.parts && (!apart || grids_last())) dependent_wait();
        if (idle) return;
        __syncwarp();  // the ring's last stage has been read by all lanes
        float *osm = join + warp * (SPW * C::STAGE / 4);
#pragma unroll
        for (int dt = 0; dt < C::DT; ++dt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    osm[(nt * 8 + 2 * c + (e & 1)) * C::OSTR + dt * 16 + r + (e >> 1) * 8] = o[dt][nt][e];
        __syncwarp();
        // lane g (and g + 16 or so) takes query head g's maximum and sum: those of row g are
        // in lane g / 2 (with r = 0) of column pair g % 2
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float m = __shfl_sync(0xffffffffu, m_ref[nt][j], (lane & 7) >> 1), l = __shfl_sync(0xffffffffu, l_run[nt][j], (lane & 7) >> 1);
                if (((lane >> 3) & (NT - 1)) == nt && (lane & 1) == j) {
                    top = m;
                    sum = l;
                }
            }
        const int g = lane & (C::NP - 1);
        const int parts = skip && !apart ? rows::live_parts((skip * BS + rows::kKeys - 1) / rows::kKeys, a.prefix.parts) : 0;
        const int64_t row = static_cast<int64_t>(s) * a.num_q_heads + h * a.group;
        if (apart && lane < a.group) a.prefix.rest_ml[row + lane] = make_float2(top, sum);
        const float2 *ml = a.prefix.ml + row + min(g, a.group - 1);
        float *pw = osm + C::NP * C::OSTR;  // [parts][NP] the prefix's weights
        auto weight = [](float m, float l, float best) { return m == -INFINITY ? (l == 0.f ? 0.f : l) : fast_exp2(m - best); };
        float all = top;
#pragma unroll 4
        for (int p = 0; p < parts; ++p) all = fmaxf(all, ml[p * a.prefix.rows].x);
        float mine = weight(top, sum, all);
        float total = mine == 0.f ? 0.f : mine * sum;
#pragma unroll 4
        for (int p = 0; p < parts; ++p) {
            const float2 x = ml[p * a.prefix.rows];
            const float f = weight(x.x, x.y, all);
            if (f != 0.f) total += f * x.y;
            if (lane < C::NP) pw[p * C::NP + g] = f;
        }
        const float inv = total != 0.f ? v_scale / total : 0.f;
        __syncwarp();
        // four head dims of a query head at a time; whole passes of the warp, for the shuffles
        const int quads = a.group * (D / 4);
        for (int i0 = 0; i0 < quads; i0 += 32) {
            const int i = min(i0 + lane, quads - 1), gi = i / (D / 4);
            if (apart) {
                if (i0 + lane < quads)
                    *reinterpret_cast<float4 *>(a.prefix.rest_o + row * D + 4 * i) = *reinterpret_cast<const float4 *>(osm + gi * C::OSTR + i % (D / 4) * 4);
                continue;
            }
            const float f0 = __shfl_sync(0xffffffffu, mine, gi), scale = __shfl_sync(0xffffffffu, inv, gi);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            auto add = [&](float f, const float4 &x) {
                if (f != 0.f) {  // an empty part's accumulator may be anything
                    v.x += f * x.x;
                    v.y += f * x.y;
                    v.z += f * x.z;
                    v.w += f * x.w;
                }
            };
            add(f0, *reinterpret_cast<const float4 *>(osm + gi * C::OSTR + i % (D / 4) * 4));
            const float *part = a.prefix.o + row * D + 4 * i;
#pragma unroll 4
            for (int p = 0; p < parts; ++p) add(pw[p * C::NP + gi], *reinterpret_cast<const float4 *>(part + p * a.prefix.rows * D));
            if (i0 + lane < quads)
                *reinterpret_cast<uint2 *>(a.out + row * D + 4 * i) = make_uint2(pack2<false>(v.x * scale, v.y * scale), pack2<false>(v.z * scale, v.w * scale));
        }
        return;
    }
    __syncthreads();  // every warp is done with the page ring
    float *osm = join;                        // [NW][NP][OSTR]
    float *msm = osm + NW * C::NP * C::OSTR;  // [NW][NP] reference
    float *lsm = msm + NW * C::NP;            // [NW][NP] sum
    float *csm = lsm + NW * C::NP;            // [NP][D] the CTA's accumulator
    float *mc = csm + C::NP * D;              // [NP] its reference
    float *lc = mc + C::NP;                   // [NP] its sum
#pragma unroll
    for (int dt = 0; dt < C::DT; ++dt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int g = nt * 8 + 2 * c + (e & 1);
                const int d = dt * 16 + r + (e >> 1) * 8;
                osm[(warp * C::NP + g) * C::OSTR + d] = o[dt][nt][e];
            }
    if (r == 0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int g = nt * 8 + 2 * c + j;
                msm[warp * C::NP + g] = m_ref[nt][j];
                lsm[warp * C::NP + g] = l_run[nt][j];
            }
    }
    __syncthreads();
    // Weights of the warps' parts, once per head.  A part that saw no token has
    // reference -infinity and sum 0 and is left out; one with a NaN in its sum
    // keeps it.
    auto weight = [](float m, float l, float top) {
        return m == -INFINITY ? (l == 0.f ? 0.f : l) : fast_exp2(m - top);
    };
    // The prefix's parts of this row and KV head, and their weights beside the
    // rest's (top, sum), which are brought up to date; the rest's own is returned.
    __shared__ float pw[SUFFIX ? rows::kMaxParts : 1][SUFFIX ? C::NP : 1];
    int parts = 0;
    if constexpr (SUFFIX) {
        if (a.prefix.parts && !a.prefix.rest_o) dependent_wait();
        if (skip && !a.prefix.rest_o) parts = rows::live_parts((skip * BS + rows::kKeys - 1) / rows::kKeys, a.prefix.parts);
    }
    const int64_t part0 = static_cast<int64_t>(s) * a.num_q_heads + h * a.group, part_stride = a.prefix.rows;
    auto with_prefix = [&](float top, float &sum) -> float {  // by thread g < group
        const float2 *ml = a.prefix.ml + part0 + tid;
        float all = top;
#pragma unroll 4
        for (int p = 0; p < parts; ++p) all = fmaxf(all, ml[p * part_stride].x);
        const float mine = weight(top, sum, all);
        sum = mine == 0.f ? 0.f : sum * mine;
#pragma unroll 4
        for (int p = 0; p < parts; ++p) {
            const float2 x = ml[p * part_stride];
            const float f = weight(x.x, x.y, all);
            if (f != 0.f) sum += f * x.y;
            pw[p][tid] = f;
        }
        return mine;
    };
    auto add_prefix = [&](int i, float4 &v) {  // four head dims of a head
        const int g = i / (D / 4);
        const float *o = a.prefix.o + part0 * D + 4 * i;
#pragma unroll 4
        for (int p = 0; p < parts; ++p) {
            const float f = pw[p][g];
            const float4 x = *reinterpret_cast<const float4 *>(o + p * part_stride * D);
            if (f != 0.f) {
                v.x += f * x.x;
                v.y += f * x.y;
                v.z += f * x.z;
                v.w += f * x.w;
            }
        }
    };
    if (tid < C::NP) {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) top = fmaxf(top, msm[w * C::NP + tid]);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float l = lsm[w * C::NP + tid], f = weight(msm[w * C::NP + tid], l, top);
            sum += f * l;
            msm[w * C::NP + tid] = f;
        }
        if constexpr (SUFFIX)
            if (ranks == 1 && tid < a.group) {
                const float mine = with_prefix(top, sum);
#pragma unroll
                for (int w = 0; w < NW; ++w) msm[w * C::NP + tid] *= mine;
            }
        mc[tid] = top;
        lc[tid] = sum;
        if constexpr (SUFFIX)
            if (a.prefix.rest_o && ranks == 1 && tid < a.group) a.prefix.rest_ml[part0 + tid] = make_float2(top, sum);
    }
    __syncthreads();
    // four head dims of a head at a time
    const int quads = num_live * (D / 4);
    auto put = [&](int i, const float4 &v, float f) {
        const uint2 w = make_uint2(pack2<false>(v.x * f, v.y * f), pack2<false>(v.z * f, v.w * f));
        *reinterpret_cast<uint2 *>(a.out + row_at(i / (D / 4)) + i % (D / 4) * 4) = w;
    };
    for (int i = tid; i < quads; i += NW * 32) {
        const int g = i / (D / 4), d = i % (D / 4) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = msm[w * C::NP + g];
            const float4 x = *reinterpret_cast<const float4 *>(osm + (w * C::NP + g) * C::OSTR + d);
            if (f != 0.f) {  // an empty part's accumulator is 0, a NaN's NaN
                v.x += f * x.x;
                v.y += f * x.y;
                v.z += f * x.z;
                v.w += f * x.w;
            }
        }
        if (ranks == 1) {
            if constexpr (SUFFIX) {
                if (a.prefix.rest_o) {
                    *reinterpret_cast<float4 *>(a.prefix.rest_o + part0 * D + 4 * i) = v;
                    continue;
                }
                add_prefix(i, v);
            }
            const float sum = lc[g];
            put(i, v, sum != 0.f ? v_scale / sum : 0.f);
        } else {
            *reinterpret_cast<float4 *>(csm + 4 * i) = v;
        }
    }
    if constexpr (SUFFIX)  // the grid is not to end before the one in front: its last CTA waits for that
        if (a.prefix.rest_o && grids_last()) dependent_wait();
    if (ranks == 1) return;

    // ---- join the CTAs: each writes its share of the output -----------------------
    cluster_arrive();
    cluster_wait();
    float *fsm = osm;  // [8][NP] the CTAs' weights over the sum (osm has been read)
    if (tid < C::NP) {
        float m[8], l[8], top = -INFINITY, sum = 0.f;
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) {
            m[k] = k < ranks ? ld_cluster(smem_addr(mc + tid), k) : -INFINITY;
            l[k] = k < ranks ? ld_cluster(smem_addr(lc + tid), k) : 0.f;
            top = fmaxf(top, m[k]);
        }
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) {
            m[k] = weight(m[k], l[k], top);
            sum += m[k] * l[k];
        }
        float mine = 1.f;
        if constexpr (SUFFIX)
            if (tid < a.group) mine = with_prefix(top, sum);
        float inv = sum != 0.f ? v_scale / sum : 0.f;
        if constexpr (SUFFIX)
            if (a.prefix.rest_o) {
                inv = 1.f;
                if (rank == 0 && tid < a.group) a.prefix.rest_ml[part0 + tid] = make_float2(top, sum);
            }
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) fsm[k * C::NP + tid] = m[k] * mine * inv;
        if constexpr (SUFFIX)
            for (int p = 0; p < parts; ++p) pw[p][tid] *= inv;
    }
    __syncthreads();
    for (int i = static_cast<int>(rank) * NW * 32 + tid; i < quads; i += static_cast<int>(ranks) * NW * 32) {
        const int g = i / (D / 4);
        uint4 x[8];
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k)
            if (k < ranks) x[k] = ld_cluster_v4(smem_addr(csm + 4 * i), k);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) {
            if (k >= ranks) break;
            const float f = fsm[k * C::NP + g];
            if (f != 0.f) {
                v.x += f * __uint_as_float(x[k].x);
                v.y += f * __uint_as_float(x[k].y);
                v.z += f * __uint_as_float(x[k].z);
                v.w += f * __uint_as_float(x[k].w);
            }
        }
        if constexpr (SUFFIX) {
            if (a.prefix.rest_o) {
                *reinterpret_cast<float4 *>(a.prefix.rest_o + part0 * D + 4 * i) = v;
                continue;
            }
            add_prefix(i, v);
        }
        put(i, v, 1.f);
    }
    // nobody leaves while another may still read its part
    cluster_arrive();
    cluster_wait();
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// Four warps to a CTA: the most CTAs whose clusters are all resident at once and
// whose warps have a page each.  An eighth of the CTAs' places is kept back:
// clusters of three, six or eight leave some of a GPC's places empty (8 rows of
// 8 heads, 16 queries each, 128K tokens: 62 us with 6, 71 with 4, 85 with 8).
// Short lists are not shared out, or little (152 rows of 8 pages 4.8 us, 5.3 with two
// CTAs, of 16 query heads 5.4 and 7.8; 72 rows of 24 pages 6.1 with two, 6.7 with six).
inline int splits_of_four_warps(int64_t rows, int pages, int resident) {
    const int most = pages < 16 ? 1 : pages < 32 && rows >= 48 ? 2 : 8;
    int splits = 1;
    for (int s : {2, 3, 4, 6, 8})
        if (s <= most && rows * s <= resident * kSms * 7 / 8 && pages >= 4 * s) splits = s;
    return splits;
}

// How whole tables are read: CTAs of a row and KV head, and warps of a CTA.  Eight
// warps, two CTAs to an SM, where they find places at once: long lists of few rows
// (one row and 8 heads, 1,000 pages: 22.5 us, 37.0 with four warps; 4 rows, 250 pages
// 11.0 and 13.7; but 69 pages 8.2 and 7.4), and one CTA to a row where there are rows
// for most places (128 rows of 19 pages 5.7 us, 6.7 with four; 256 of 94 24.2, 25.1 by
// two CTAs of four).  Of more rows four CTAs to an SM hide more of each other (512 of 25
// pages 15.7 and 14.1).  `live`: rows of queries.
struct Spread {
    int splits, warps;
};
inline int64_t places_of_eight_warps(int resident, int live) { return live <= 8 ? resident / 2 * kSms * 7 / 8 : 0; }
inline Spread spread_of_tables(int64_t rows, int pages, int resident, int live) {
    const int64_t places = places_of_eight_warps(resident, live);
    if (rows * 8 <= places && pages >= 128) return {8, 8};
    if (rows <= places && (rows >= 200 ? pages >= 16 : rows >= 96 && pages >= 16 && pages < 40)) return {1, 8};
    return {splits_of_four_warps(rows, pages, resident), 4};
}

// Steps of a warp's ring.  Up to 8 query heads at head dim 128 one step, 32 KB
// to a CTA and four CTAs to an SM, against two steps and three CTAs: 112 and 116
// us over 64 sequences of 4K-32K tokens, 60 and 63 with E4M3 pages (512 clusters
// of one CTA: four to an SM have places for all of them).  Groups above 8 need
// so many registers that fewer CTAs fit, and take the memory: 64 KB for three
// CTAs, 96 KB for two.  Head dim 64: two steps, 32 KB mostly.
template <int D, int BS, bool FP8, int NT>
constexpr int stages_per_warp() {
    if (D == 64) return 2;
    if (NT == 1) return 1;
    constexpr int ppi = (FP8 && BS == 16) ? 2 : 1;
    constexpr int stage = 2 * ppi * BS * D * (FP8 ? 1 : 2);
    constexpr int spw = (BS == 16 && !FP8 ? 64 : 96) * 1024 / (4 * stage);
    return spw < 1 ? 1 : spw;
}

template <int D, int BS, bool FP8, int NT, int NW, int MODE>
static pa_status launch_attend(const CUtensorMap &tk, const CUtensorMap &tv, const Args &a0, int num_rows,
                               int splits, cudaStream_t stream) {
    constexpr int SPW = stages_per_warp<D, BS, FP8, NT>();
    constexpr bool CHOOSE = MODE == kChoose;
    using C = Shape<D, BS, FP8, NT, NW, SPW>;
    // The choice works where the ring will be: copies of bounds, then keys.  Long
    // shares take more shared memory than the ring.
    Args a = a0;
    int smem = C::SMEM;
    if constexpr (CHOOSE) {
        const int keys = key_bytes(a.select.max_blocks, splits);
        a.select.stages = copy_bytes(NW * 32, D, kMaxStages) + keys <= C::SMEM - 1024 ? kMaxStages : 2;
        smem = std::max(smem, 1024 + copy_bytes(NW * 32, D, a.select.stages) + keys);
    }
    constexpr int kMostSmem = CHOOSE ? std::max(C::SMEM, 1024 + copy_bytes(NW * 32, D, 2) + (kMaxKeys + 4) * 4) : C::SMEM;
    auto kern = attend_kernel<D, BS, FP8, NT, NW, SPW, MODE>;
    static std::atomic<uint64_t> raised{0};
    pa_status st = raise_smem_limit(reinterpret_cast<const void *>(kern), kMostSmem, raised);
    if (st != PA_OK) return st;
    const int heads = MODE == kSuffixHeads ? (a.num_kv_heads + NW - 1) / NW : a.num_kv_heads;
    return cuda_check(launch_dependent(kern, dim3(splits, heads, num_rows), NW * 32, smem, splits, stream, tk, tv, a),
                      "sparse decode launch");
}

// Eight warps to a CTA: up to 8 query heads, and not for lists that come with the call.
template <int D, int BS, bool FP8, int MODE>
static pa_status launch_group(const CUtensorMap &tk, const CUtensorMap &tv, const Args &a, int num_rows, int splits,
                              int warps, cudaStream_t stream, int live) {
    if (live > 8) return launch_attend<D, BS, FP8, 2, 4, MODE>(tk, tv, a, num_rows, splits, stream);
    if constexpr (MODE == kChoose || MODE == kSuffix || MODE == kRows)
        if (warps == 8) return launch_attend<D, BS, FP8, 1, 8, MODE>(tk, tv, a, num_rows, splits, stream);
    return launch_attend<D, BS, FP8, 1, 4, MODE>(tk, tv, a, num_rows, splits, stream);
}

// `live`: rows of queries to a cluster (the group, but for kRows).
template <int MODE>
static pa_status launch_any(int head_dim, int block_size, bool fp8, const CUtensorMap &tk, const CUtensorMap &tv,
                            const Args &a, int num_rows, int splits, int warps, cudaStream_t stream, int live) {
    auto shape = [&](auto d, auto bs) {
        return fp8 ? launch_group<d.value, bs.value, true, MODE>(tk, tv, a, num_rows, splits, warps, stream, live)
                   : launch_group<d.value, bs.value, false, MODE>(tk, tv, a, num_rows, splits, warps, stream, live);
    };
    using I64 = std::integral_constant<int, 64>;
    using I128 = std::integral_constant<int, 128>;
    using I16 = std::integral_constant<int, 16>;
    using I32 = std::integral_constant<int, 32>;
    if (head_dim == 128) return block_size == 16 ? shape(I128{}, I16{}) : shape(I128{}, I32{});
    return block_size == 16 ? shape(I64{}, I16{}) : shape(I64{}, I32{});
}

}  // namespace sparse
}  // namespace pa
