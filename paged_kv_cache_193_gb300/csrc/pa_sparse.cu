// Which pages a decode step attends to: int8 bounds of every full page's keys
// (block summary), and the choice of the pages whose bound of q . k is
// largest (sparse select).  The pages motivate contexts of 128K tokens ("vLLM
// PagedAttention Optimization: Complete Step-by-Step Tuning Guide", Step 1)
// and attend to all of them; attending to a chosen part is this library's own.
//
// Mathematics.  For a page's keys k_t (t over its tokens) let hi_d = max_t
// k_t,d and lo_d = min_t k_t,d.  Then for any query q,
//   q . k_t <= sum_d max(q_d hi_d, q_d lo_d).
// hi, lo and q are held as whole numbers of at most 127 times a power of two
// shared by the page and head (by the query head), so the bound is a whole
// number, the sum has no rounding and no order, and two pages compare the
// same way on any machine.  Eight bits with a shared power of two are coarse
// (steps of 1/64 to 1/127 of the largest value) but only rank pages.
#include <cooperative_groups.h>

#include "pa_sparse.cuh"

namespace pa {
namespace sparse {

namespace cg = cooperative_groups;

// Least exponent e in [kMinExp, kMaxExp] with amax <= 127 * 2^e.
__device__ __forceinline__ int shared_exponent(float amax) {
    if (!(amax > 0.f)) return kMinExp;
    int x;
    const float part = frexpf(amax, &x);
    const int e = x - 7 + (part * 128.f > 127.f ? 1 : 0);
    return max(kMinExp, min(kMaxExp, e));
}

// 2^e for e in [-126, 127], exactly.
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((e + 127) << 23); }

// rint(x * 2^-e) held to +-127 (above only where e was clamped to kMaxExp)
__device__ __forceinline__ int to_int8(float x, float inv_unit) {
    return max(-127, min(127, __float2int_rn(x * inv_unit)));
}

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
    unsigned int *err;
};

// A CTA looks at 32 slots; each of its warps takes (completed page, head)
// items in turn.  A lane reads 16-byte pieces of the page's rows, all before
// the first is used.
template <int D, int BS, bool FP8>
__global__ void __launch_bounds__(256) summary_kernel(const SummaryArgs a) {
    constexpr int ELEM = FP8 ? 1 : 2;
    constexpr int EPL = 16 / ELEM;       // elements of a lane's piece
    constexpr int LPR = D / EPL;         // lanes to a row
    constexpr int RPL = 32 / LPR;        // rows per load of the warp
    constexpr int LOADS = BS / RPL;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int token = blockIdx.x * 32 + lane;
    int32_t slot = token < a.num_tokens ? a.slots[token] : -1;
    if (slot >= a.num_slots) {
        if (warp == 0) set_device_error(a.err, PA_DEVERR_BAD_SLOT);
        slot = -1;
    }
    uint32_t ends = __ballot_sync(0xffffffffu, slot >= 0 && slot % BS == BS - 1);
    const int items = __popc(ends) * a.num_kv_heads;
    for (int it = warp; it < items; it += 8) {
        const int nth = it / a.num_kv_heads, h = it - nth * a.num_kv_heads;
        const int from = __fns(ends, 0, nth + 1);
        const int64_t blk = __shfl_sync(0xffffffffu, slot, from) / BS;
        const int64_t row = blk * a.num_kv_heads + h;
        const uint8_t *src = a.k_cache + row * (BS * D * ELEM) + lane * 16;
        uint4 w[LOADS];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) w[i] = *reinterpret_cast<const uint4 *>(src + i * 512);
        float hi[EPL], lo[EPL];
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
            hi[e] = -INFINITY;
            lo[e] = INFINITY;
        }
        bool odd = false;  // an infinity or NaN among the keys
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                if constexpr (FP8) {
                    uint32_t l2, h2;
                    e4m3x4_to_f16x2x2(u[p], l2, h2);
                    const float2 f0 = __half22float2(*reinterpret_cast<__half2 *>(&l2));
                    const float2 f1 = __half22float2(*reinterpret_cast<__half2 *>(&h2));
                    const float x[4] = {f0.x, f0.y, f1.x, f1.y};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        odd |= !(fabsf(x[e]) < INFINITY);
                        hi[4 * p + e] = fmaxf(hi[4 * p + e], x[e]);
                        lo[4 * p + e] = fminf(lo[4 * p + e], x[e]);
                    }
                } else {
                    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u[p]));
                    odd |= !(fabsf(f.x) < INFINITY) || !(fabsf(f.y) < INFINITY);
                    hi[2 * p] = fmaxf(hi[2 * p], f.x);
                    lo[2 * p] = fminf(lo[2 * p], f.x);
                    hi[2 * p + 1] = fmaxf(hi[2 * p + 1], f.y);
                    lo[2 * p + 1] = fminf(lo[2 * p + 1], f.y);
                }
            }
        }
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
#pragma unroll
            for (int m = LPR; m < 32; m <<= 1) {
                hi[e] = fmaxf(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], m));
                lo[e] = fminf(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], m));
            }
            amax = fmaxf(amax, fmaxf(fabsf(hi[e]), fabsf(lo[e])));
        }
#pragma unroll
        for (int m = 1; m < LPR; m <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
        odd = __any_sync(0xffffffffu, odd);
        const int ex = odd ? kOddExp : shared_exponent(amax);
        const float inv = odd ? 0.f : power_of_two(-ex);
        if (lane < 2 * LPR) {  // the first lanes write the largest, the next the least
            int8_t *dst = a.summary + row * (2 * D) + lane * EPL;
            uint32_t out[EPL / 4];
#pragma unroll
            for (int e = 0; e < EPL; e += 4) {
                uint32_t v = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const float x = lane < LPR ? hi[e + b] : lo[e + b];
                    v |= static_cast<uint32_t>((odd ? 0 : to_int8(x, inv)) & 0xff) << (8 * b);
                }
                out[e / 4] = v;
            }
#pragma unroll
            for (int e = 0; e < EPL / 4; ++e) reinterpret_cast<uint32_t *>(dst)[e] = out[e];
        }
        if (lane == 0) a.exponents[row] = static_cast<int8_t>(ex);
    }
}

// ---------------------------------------------------------------------------
// select
// ---------------------------------------------------------------------------

struct SelectArgs {
    const __nv_bfloat16 *q;
    const int8_t *summary;
    const int8_t *exponents;
    const int32_t *block_tables;
    const int32_t *context_lens;
    int32_t *selected;  // [num_rows][num_kv_heads][top_k]
    int32_t *counts;    // [num_rows][num_kv_heads]
    int max_blocks, num_blocks, num_kv_heads, group, block_size;
    int top_k, sink, recent;
    int keys_per_cta;  // shared-memory room for keys
    unsigned int *err;
};

// fp32 -> unsigned with the same order
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

constexpr int kSelThreads = 256;

// One cluster of CTAs per (row, KV head): each scores its share of the
// candidate pages into its own shared memory, the cluster finds the score of
// the last page to be taken by a radix search (eight bits at a time, the
// CTAs' histograms summed over distributed shared memory), and each CTA
// writes the chosen pages of its share in order.
template <int D>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectArgs a) {
    constexpr int LPB = 2 * D / 16;  // lanes to a page's summary
    constexpr int PPW = 32 / LPB;    // pages per load of the warp
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ __align__(16) uint32_t qi[16][2 * D / 4];
    __shared__ float qunit[16];
    __shared__ uint32_t hist[2][256];
    __shared__ uint32_t total[256];
    __shared__ uint32_t pick[2];
    __shared__ uint32_t mine[2];
    __shared__ uint32_t warp_sum[2][kSelThreads / 32];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = cluster.block_rank(), ranks = cluster.num_blocks();
    const int h = blockIdx.y, t = blockIdx.z;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t out_row = static_cast<int64_t>(t) * a.num_kv_heads + h;
    int32_t *out = a.selected + out_row * a.top_k;

    int n = a.context_lens[t];
    if (n > a.max_blocks * a.block_size) {
        if (tid == 0 && rank == 0 && h == 0) set_device_error(a.err, PA_DEVERR_BAD_CONTEXT);
        n = a.max_blocks * a.block_size;
    }
    const int nb = n > 0 ? (n + a.block_size - 1) / a.block_size : 0;
    const int count = min(nb, a.top_k);
    // entries behind the chosen ones, and the count
    for (int i = count + rank * kSelThreads + tid; i < a.top_k; i += ranks * kSelThreads) out[i] = -1;
    if (rank == 0 && tid == 0) a.counts[out_row] = count;
    if (nb <= a.top_k) {
        for (int i = rank * kSelThreads + tid; i < count; i += ranks * kSelThreads) out[i] = i;
        return;  // the same for every CTA of the cluster
    }
    const int want = a.top_k - a.sink - a.recent;  // pages to take from the candidates
    for (int i = rank * kSelThreads + tid; i < a.sink; i += ranks * kSelThreads) out[i] = i;
    for (int i = rank * kSelThreads + tid; i < a.recent; i += ranks * kSelThreads)
        out[a.top_k - a.recent + i] = nb - a.recent + i;
    if (want == 0) return;

    // the group's queries as whole numbers: positive parts, then negative
    for (int g = warp; g < a.group; g += kSelThreads / 32) {
        const __nv_bfloat16 *qg = a.q + (out_row * a.group + g) * D + lane * (D / 32);
        float x[D / 32], amax = 0.f;
        bool odd = false;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            x[i] = __bfloat162float(qg[i]);
            odd |= !(fabsf(x[i]) < INFINITY);
            amax = fmaxf(amax, fabsf(x[i]));
        }
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
        odd = __any_sync(0xffffffffu, odd);
        const int e = odd ? kMinExp : shared_exponent(amax);
        const float inv = power_of_two(-e);
        int8_t *dst = reinterpret_cast<int8_t *>(qi[g]);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const int r = odd ? 0 : to_int8(x[i], inv);
            dst[lane * (D / 32) + i] = static_cast<int8_t>(max(r, 0));
            dst[D + lane * (D / 32) + i] = static_cast<int8_t>(min(r, 0));
        }
        if (lane == 0) qunit[g] = power_of_two(e);
    }
    __syncthreads();

    // ---- scores of this CTA's share of the candidates -------------------------
    const int ncand = nb - a.sink - a.recent;
    const int per = (ncand + ranks - 1) / ranks;
    const int c0 = rank * per, c1 = min(ncand, c0 + per);
    const int have = max(0, c1 - c0);
    const int32_t *table = a.block_tables + static_cast<int64_t>(t) * a.max_blocks + a.sink;
    const int part = lane % LPB;
    for (int base = c0 + warp * 32; base < c1; base += kSelThreads) {
        int32_t blk = 0;
        int ex = kMinExp;
        bool bad = false;
        if (base + lane < c1) {
            blk = table[base + lane];
            if (blk < 0 || blk >= a.num_blocks) {
                set_device_error(a.err, PA_DEVERR_BAD_BLOCK);
                bad = true;
                blk = 0;
            }
            ex = a.exponents[static_cast<int64_t>(blk) * a.num_kv_heads + h];
        }
        float score = -INFINITY;
#pragma unroll 4
        for (int i = 0; i < 32; i += PPW) {
            const int32_t b = __shfl_sync(0xffffffffu, blk, i + lane / LPB);
            const uint4 w = __ldg(reinterpret_cast<const uint4 *>(
                a.summary + (static_cast<int64_t>(b) * a.num_kv_heads + h) * (2 * D) + part * 16));
            float best = -INFINITY;
            for (int g = 0; g < a.group; ++g) {
                const uint4 r = *reinterpret_cast<const uint4 *>(&qi[g][part * 4]);
                int dot = __dp4a(static_cast<int>(w.x), static_cast<int>(r.x), 0);
                dot = __dp4a(static_cast<int>(w.y), static_cast<int>(r.y), dot);
                dot = __dp4a(static_cast<int>(w.z), static_cast<int>(r.z), dot);
                dot = __dp4a(static_cast<int>(w.w), static_cast<int>(r.w), dot);
#pragma unroll
                for (int m = 1; m < LPB; m <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
                best = fmaxf(best, static_cast<float>(dot) * qunit[g]);
            }
            const float mine_now = __shfl_sync(0xffffffffu, best, (lane % PPW) * LPB);
            if (lane >= i && lane < i + PPW) score = mine_now;
        }
        if (base + lane < c1) {
            score = bad ? -INFINITY : ex == kOddExp ? INFINITY : score * power_of_two(ex);
            keys[base + lane - c0] = order_key(score);
        }
    }

    // ---- the key of the last page taken ---------------------------------------
    uint32_t prefix = 0;
    uint32_t left = want;  // pages still to be found among keys with this prefix
    for (int pass = 0; pass < 4; ++pass) {
        uint32_t *hs = hist[pass & 1];
        hs[tid] = 0;
        __syncthreads();
        const int shift = 24 - 8 * pass;
        for (int i = tid; i < have; i += kSelThreads) {
            const uint32_t key = keys[i];
            if (pass == 0 || (key >> (shift + 8)) == prefix) atomicAdd(&hs[(key >> shift) & 255u], 1u);
        }
        cluster.sync();
        uint32_t sum = 0;
        for (int r = 0; r < ranks; ++r) sum += cluster.map_shared_rank(hs, r)[tid];
        total[tid] = sum;
        __syncthreads();
        if (warp == 0) {  // from the top, the bin that holds the left-th key
            uint32_t v[8], s = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = total[255 - (lane * 8 + i)];
                s += v[i];
            }
            uint32_t before = s;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, before, m);
                if (lane >= m) before += o;
            }
            before -= s;
            if (before < left && before + s >= left) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (before < left && before + v[i] >= left) {
                        pick[0] = 255 - (lane * 8 + i);
                        pick[1] = left - before;
                        break;
                    }
                    before += v[i];
                }
            }
        }
        __syncthreads();
        prefix = (prefix << 8) | pick[0];
        left = pick[1];
        __syncthreads();
    }
    // now: every key above `prefix` is taken, and the first `left` equal to it

    // ---- how many each CTA takes, and where it writes -------------------------
    uint32_t above = 0, equal = 0;
    for (int i = tid; i < have; i += kSelThreads) {
        above += keys[i] > prefix;
        equal += keys[i] == prefix;
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
        warp_sum[0][warp] = above;
        warp_sum[1][warp] = equal;
    }
    __syncthreads();
    if (tid == 0) {
        uint32_t x = 0, y = 0;
        for (int w = 0; w < kSelThreads / 32; ++w) {
            x += warp_sum[0][w];
            y += warp_sum[1][w];
        }
        mine[0] = x;
        mine[1] = y;
    }
    cluster.sync();
    uint32_t above0 = 0, equal0 = 0;  // of the CTAs before this one
    for (int r = 0; r < rank; ++r) {
        above0 += cluster.map_shared_rank(mine, r)[0];
        equal0 += cluster.map_shared_rank(mine, r)[1];
    }
    for (int base = 0; base < have; base += kSelThreads) {
        const int i = base + tid;
        const uint32_t key = i < have ? keys[i] : 0;
        const bool is_above = i < have && key > prefix, is_equal = i < have && key == prefix;
        const uint32_t ma = __ballot_sync(0xffffffffu, is_above), me = __ballot_sync(0xffffffffu, is_equal);
        __syncthreads();  // the sums of the step before have been read
        if (lane == 0) {
            warp_sum[0][warp] = __popc(ma);
            warp_sum[1][warp] = __popc(me);
        }
        __syncthreads();
        uint32_t xa = above0, xe = equal0, ta = 0, te = 0;
#pragma unroll
        for (int w = 0; w < kSelThreads / 32; ++w) {
            if (w < warp) {
                xa += warp_sum[0][w];
                xe += warp_sum[1][w];
            }
            ta += warp_sum[0][w];
            te += warp_sum[1][w];
        }
        const uint32_t below = (1u << lane) - 1u;
        xa += __popc(ma & below);
        xe += __popc(me & below);
        if (is_above || (is_equal && xe < left))
            out[a.sink + xa + min(xe, left)] = a.sink + c0 + i;
        above0 += ta;
        equal0 += te;
    }
    cluster.sync();  // nobody leaves while another may still read its sums
}

template <int D>
static pa_status launch_select(const SelectArgs &a0, int num_rows, cudaStream_t stream) {
    SelectArgs a = a0;
    // enough CTAs to fill the machine, and no more than the pages can use
    const int64_t rows = static_cast<int64_t>(num_rows) * a.num_kv_heads;
    int ranks = 1;
    while (ranks < 8 && rows * ranks < 2 * 152 && a.max_blocks > 128 * ranks) ranks *= 2;
    while (ranks < 8 && a.max_blocks > 32768 * ranks) ranks *= 2;
    a.keys_per_cta = (a.max_blocks + ranks - 1) / ranks;
    const size_t smem = static_cast<size_t>(a.keys_per_cta) * 4;
    auto kern = select_kernel<D>;
    static std::atomic<uint64_t> raised{0};
    pa_status st = raise_smem_limit(reinterpret_cast<const void *>(kern), kMaxSelectSmem, raised);
    if (st != PA_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ranks, a.num_kv_heads, num_rows);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_check(cudaLaunchKernelEx(&cfg, kern, a), "sparse select launch");
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
    if (max_blocks > kMaxTableBlocks)
        return fail(PA_ERR_UNSUPPORTED, "max_blocks_per_seq %d (supported: up to %d)", max_blocks, kMaxTableBlocks);
    return PA_OK;
}

pa_status run_select(const void *q, const int8_t *summary, const int8_t *exponents,
                     const int32_t *block_tables, int max_blocks, const int32_t *context_lens,
                     int num_rows, int num_q_heads, int num_kv_heads, int head_dim, int num_blocks,
                     int block_size, int top_k, int sink, int recent, int32_t *selected,
                     int32_t *counts, cudaStream_t stream) {
    unsigned int *err = device_error_word();
    if (!err) return fail(PA_ERR_CUDA, "cannot resolve the device error word");
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
    a.err = err;
    return head_dim == 128 ? launch_select<128>(a, num_rows, stream) : launch_select<64>(a, num_rows, stream);
}

template <int D, int BS>
static void launch_summary(const SummaryArgs &a, bool fp8, unsigned grid, cudaStream_t stream) {
    if (fp8)
        summary_kernel<D, BS, true><<<grid, 256, 0, stream>>>(a);
    else
        summary_kernel<D, BS, false><<<grid, 256, 0, stream>>>(a);
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
    const unsigned grid = (static_cast<unsigned>(num_tokens) + 31) / 32;
    if (head_dim == 128)
        block_size == 16 ? launch_summary<128, 16>(a, fp8, grid, stream)
                         : launch_summary<128, 32>(a, fp8, grid, stream);
    else
        block_size == 16 ? launch_summary<64, 16>(a, fp8, grid, stream)
                         : launch_summary<64, 32>(a, fp8, grid, stream);
    return cuda_check(cudaGetLastError(), "block summary launch");
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
    return run_select(q, summary, exponents, block_tables, max_blocks_per_seq, context_lens, num_rows,
                      num_q_heads, num_kv_heads, head_dim, num_blocks, block_size, top_k, sink_blocks,
                      recent_blocks, selected, counts, stream);
}

}  // extern "C"
