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
#include "pa_sparse.cuh"

namespace pa {
namespace sparse {

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
    unsigned int *err;
};

// fp32 -> unsigned with the same order
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

// Four signed bytes of a word as exact fp16 pairs: even = bytes 0 and 2, odd =
// bytes 1 and 3.  0x6400 | (x + 128) is the fp16 value 1152 + x.
__device__ __forceinline__ void int8x4_to_f16(uint32_t w, uint32_t &even, uint32_t &odd) {
    const uint32_t e = (w & 0x00ff00ffu) ^ 0x64806480u;
    const uint32_t o = ((w >> 8) & 0x00ff00ffu) ^ 0x64806480u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    const __half2 he = __hsub2(*reinterpret_cast<const __half2 *>(&e), off);
    const __half2 ho = __hsub2(*reinterpret_cast<const __half2 *>(&o), off);
    even = *reinterpret_cast<const uint32_t *>(&he);
    odd = *reinterpret_cast<const uint32_t *>(&ho);
}

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 4 * kSelThreads;  // of a histogram: four to a thread
constexpr int kBinBits = 10;
constexpr int kListMax = kSelThreads;   // keys that are ranked one against another

// One cluster of CTAs per (row, KV head): each scores its share of the
// candidate pages into its own shared memory, the cluster finds the score of
// the last page to be taken, and each CTA writes the chosen pages of its share
// in order.
//
// Scores: 16 pages x 8 query heads x 16 bounds are one m16n8k16 product in
// fp16 (every int8 value is one) with fp32 sums of at most 2^22: exact.  A
// lane reads 16-byte pieces of a page's bounds straight from global memory
// into the product's A fragment; the order of the sum is free, so the query
// takes the order that the bytes lie in.
// Choice: a histogram of the keys over their own range, the bin that holds
// the last page to be taken, and, once few keys are left in the bin, their
// ranks among one another.
template <int D, int NT>
__global__ void __launch_bounds__(kSelThreads, 2) select_kernel(const SelectArgs a) {
    constexpr int PIECES = 2 * D / 64;  // 16-byte pieces of a page that a lane reads
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ __align__(16) uint32_t hist[2][kBins];
    __shared__ uint32_t list[kListMax], ranked[kListMax];
    __shared__ uint32_t list_len;
    __shared__ uint32_t range_s[2];      // least and largest key of the CTA
    __shared__ uint32_t warp_s[2][kSelWarps];
    __shared__ uint32_t pick[3];
    __shared__ uint32_t taken[2];        // pages above, and equal to, the last key
    const int rank = static_cast<int>(cluster_rank()), ranks = static_cast<int>(cluster_size());
    const int h = blockIdx.y, t = blockIdx.z;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = lane >> 2, c = lane & 3;
    const int64_t out_row = static_cast<int64_t>(t) * a.num_kv_heads + h;
    int32_t *out = a.selected + out_row * a.top_k;
    auto sync_all = [&]() {
        if (ranks > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
    };

    // the group's queries, as they are needed below: lane (r, c) holds 16-dim
    // pieces c, c + 4, ... of head r (and r + 8)
    constexpr int QP = D / 64;  // pieces of a query head that a lane holds
    uint4 qraw[NT][QP][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int g = nt * 8 + r;
        const uint4 *qg = reinterpret_cast<const uint4 *>(a.q + (out_row * a.group + min(g, a.group - 1)) * D);
#pragma unroll
        for (int i = 0; i < QP; ++i) {
            qraw[nt][i][0] = __ldg(qg + 2 * (c + 4 * i));
            qraw[nt][i][1] = __ldg(qg + 2 * (c + 4 * i) + 1);
        }
    }
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

    const int ncand = nb - a.sink - a.recent;
    const int per = ((ncand + ranks - 1) / ranks + 15) & ~15;
    const int c0 = min(ncand, rank * per), c1 = min(ncand, c0 + per);
    const int have = c1 - c0;
    const int32_t *table = a.block_tables + static_cast<int64_t>(t) * a.max_blocks + a.sink;
    int base = c0 + warp * 16;
    const int in16 = lane & 15;
    int32_t next_blk = base + in16 < c1 ? __ldg(table + base + in16) : -1;

    if (tid == 0) {
        range_s[0] = 0xffffffffu;
        range_s[1] = 0;
        list_len = 0;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
        reinterpret_cast<uint4 *>(hist[i])[tid] = make_uint4(0, 0, 0, 0);

    // queries as whole numbers: B fragments of their positive (for the largest
    // keys) and negative parts (for the least)
    uint32_t qf[NT][PIECES][4][2];
    float unit[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float x[QP][16], amax = 0.f;
        bool odd = false;
#pragma unroll
        for (int i = 0; i < QP; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint4 &u = qraw[nt][i][j / 4];
                const uint32_t w = j % 4 == 0 ? u.x : j % 4 == 1 ? u.y : j % 4 == 2 ? u.z : u.w;
                const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
                x[i][2 * j] = f.x;
                x[i][2 * j + 1] = f.y;
                odd |= !(fabsf(f.x) < INFINITY) || !(fabsf(f.y) < INFINITY);
                amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
        const uint32_t votes = __ballot_sync(0xffffffffu, odd);
        odd = (votes >> (lane & 28)) & 15u;
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int e = odd ? kMinExp : shared_exponent(amax);
        const float inv = power_of_two(-e), mine = power_of_two(e);
#pragma unroll
        for (int i = 0; i < QP; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float v[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    v[u] = odd ? 0.f : static_cast<float>(to_int8(x[i][4 * j + u], inv));
                qf[nt][i][j][0] = pack2<true>(fmaxf(v[0], 0.f), fmaxf(v[2], 0.f));
                qf[nt][i][j][1] = pack2<true>(fmaxf(v[1], 0.f), fmaxf(v[3], 0.f));
                qf[nt][QP + i][j][0] = pack2<true>(fminf(v[0], 0.f), fminf(v[2], 0.f));
                qf[nt][QP + i][j][1] = pack2<true>(fminf(v[1], 0.f), fminf(v[3], 0.f));
            }
#pragma unroll
        for (int j = 0; j < 2; ++j) unit[nt][j] = __shfl_sync(0xffffffffu, mine, (2 * c + j) * 4);
    }
    __syncthreads();

    // ---- scores of this CTA's share of the candidates -------------------------
    uint32_t kmin = 0xffffffffu, kmax = 0;
    for (; base < c1; base += 16 * kSelWarps) {
        int32_t blk = next_blk;
        const int ahead = base + 16 * kSelWarps + in16;
        next_blk = ahead < c1 ? __ldg(table + ahead) : -1;
        const bool bad = blk < 0 || blk >= a.num_blocks;
        if (bad) {
            if (base + in16 < c1) set_device_error(a.err, PA_DEVERR_BAD_BLOCK);
            blk = 0;
        }
        const int64_t row = static_cast<int64_t>(blk) * a.num_kv_heads + h;
        int ex = a.exponents[row];
        if (bad) ex = kOddExp + 1;
        uint4 w[2][PIECES];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int64_t prow = __shfl_sync(0xffffffffu, row, r + 8 * p);
            const uint4 *src = reinterpret_cast<const uint4 *>(a.summary + prow * (2 * D)) + c;
#pragma unroll
            for (int i = 0; i < PIECES; ++i) w[p][i] = __ldg(src + 4 * i);
        }
        float acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                auto word = [&](const uint4 &u) { return j == 0 ? u.x : j == 1 ? u.y : j == 2 ? u.z : u.w; };
                uint32_t a0, a1, a2, a3;
                int8x4_to_f16(word(w[0][i]), a0, a2);
                int8x4_to_f16(word(w[1][i]), a1, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma16816<true>(acc[nt], a0, a1, a2, a3, qf[nt][i][j][0], qf[nt][i][j][1]);
            }
        float s0 = -INFINITY, s1 = -INFINITY;  // pages r and r + 8
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (nt * 8 + 2 * c + j < a.group) {
                    s0 = fmaxf(s0, acc[nt][j] * unit[nt][j]);
                    s1 = fmaxf(s1, acc[nt][2 + j] * unit[nt][j]);
                }
#pragma unroll
        for (int m = 1; m < 4; m <<= 1) {
            s0 = fmaxf(s0, __shfl_xor_sync(0xffffffffu, s0, m));
            s1 = fmaxf(s1, __shfl_xor_sync(0xffffffffu, s1, m));
        }
        const int page = r + 8 * (c & 1);
        ex = __shfl_sync(0xffffffffu, ex, page);
        if (c < 2 && base + page < c1) {
            const float score = ex > kOddExp ? -INFINITY : ex == kOddExp ? INFINITY : (c ? s1 : s0) * power_of_two(ex);
            const uint32_t key = order_key(score);
            keys[base + page - c0] = key;
            kmin = min(kmin, key);
            kmax = max(kmax, key);
        }
    }
    kmin = __reduce_min_sync(0xffffffffu, kmin);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    if (lane == 0) {
        atomicMin(&range_s[0], kmin);
        atomicMax(&range_s[1], kmax);
    }
    sync_all();

    // ---- the key of the last page taken ---------------------------------------
    uint32_t low = range_s[0], high = range_s[1];
    for (int k = 1; k < ranks; ++k) {
        const uint32_t other = static_cast<uint32_t>((rank + k) % ranks);
        low = min(low, ld_cluster_u32(smem_addr(&range_s[0]), other));
        high = max(high, ld_cluster_u32(smem_addr(&range_s[1]), other));
    }
    uint32_t span = high - low;  // keys looked at: low .. low + span
    int shift = max(0, 32 - __clz(span) - kBinBits);
    uint32_t left = want;  // pages still to be found among them
    uint32_t last;         // the last key taken, by the `left` first pages that have it
    for (int pass = 0;; ++pass) {
        uint32_t *hs = hist[pass & 1];
        for (int i = tid; i < have; i += kSelThreads) {
            const uint32_t d = keys[i] - low;  // of a key below: past span
            if (d <= span) atomicAdd(&hs[d >> shift], 1u);
        }
        sync_all();
        // four bins to a thread, from the top
        const uint32_t at = smem_addr(hs) + (kSelThreads - 1 - tid) * 16;
        uint4 v = make_uint4(0, 0, 0, 0);
        for (int k = 0; k < ranks; ++k) {
            const uint4 o = ranks > 1 ? ld_cluster_v4(at, k) : lds128(at);
            v.x += o.x;
            v.y += o.y;
            v.z += o.z;
            v.w += o.w;
        }
        const uint32_t sum = v.x + v.y + v.z + v.w;
        uint32_t before = sum;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, before, m);
            if (lane >= m) before += o;
        }
        if (lane == 31) warp_s[0][warp] = before;
        before -= sum;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kSelWarps; ++w)
            if (w < warp) before += warp_s[0][w];
        if (before < left && before + sum >= left) {
            const uint32_t bins[4] = {v.w, v.z, v.y, v.x};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (before < left && before + bins[k] >= left) {
                    pick[0] = kBins - 1 - (4 * tid + k);
                    pick[1] = left - before;
                    pick[2] = bins[k];
                }
                before += bins[k];
            }
        }
        // the histogram of the pass before: every CTA has read it
        if (pass > 0) reinterpret_cast<uint4 *>(hist[(pass + 1) & 1])[tid] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        low += pick[0] << shift;
        left = pick[1];
        const uint32_t found = pick[2];
        span = (1u << shift) - 1u;
        if (found <= kListMax) {
            // the bin's keys, gathered in the first CTA, ranked by every CTA
            for (int i = tid; i < have; i += kSelThreads) {
                const uint32_t key = keys[i];
                if (key - low <= span) {
                    if (ranks > 1)
                        st_cluster_u32(smem_addr(list) + 4 * atom_add_cluster(smem_addr(&list_len), 0, 1u), 0, key);
                    else
                        list[atomicAdd(&list_len, 1u)] = key;
                }
            }
            sync_all();
            const uint32_t key = tid >= found ? 0u : ranks > 1 ? ld_cluster_u32(smem_addr(list) + 4 * tid, 0) : list[tid];
            ranked[tid] = key;
            __syncthreads();
            uint32_t greater = 0, equal = 0;
            for (uint32_t j = 0; j < found; ++j) {
                greater += ranked[j] > key;
                equal += ranked[j] == key;
            }
            if (tid < found && greater < left && greater + equal >= left) {
                pick[0] = key;  // by every page that has it: the same values
                pick[1] = left - greater;
            }
            __syncthreads();
            last = pick[0];
            left = pick[1];
            break;
        }
        if (shift == 0) {  // one key, more often than the list is long
            last = low;
            break;
        }
        shift = max(0, shift - kBinBits);
    }

    // ---- every key above `last`, and the first `left` equal to it --------------
    const int seg = ((have + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int i0 = min(have, warp * seg), i1 = min(have, i0 + seg);
    uint32_t above = 0, equal = 0;
    for (int i = i0 + lane; i < i1; i += 32) {
        above += keys[i] > last;
        equal += keys[i] == last;
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
        warp_s[0][warp] = above;
        warp_s[1][warp] = equal;
    }
    __syncthreads();
    uint32_t xa = 0, xe = 0;  // taken, and equal, before this warp's
    if (ranks > 1) {
        if (tid == 0) {
            uint32_t sa = 0, se = 0;
            for (int w = 0; w < kSelWarps; ++w) {
                sa += warp_s[0][w];
                se += warp_s[1][w];
            }
            taken[0] = sa;
            taken[1] = se;
        }
        sync_all();
        for (int k = 0; k < rank; ++k) {
            xa += ld_cluster_u32(smem_addr(&taken[0]), k);
            xe += ld_cluster_u32(smem_addr(&taken[1]), k);
        }
    }
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w)
        if (w < warp) {
            xa += warp_s[0][w];
            xe += warp_s[1][w];
        }
    const uint32_t below = (1u << lane) - 1u;
    for (int b = i0; b < i1; b += 32) {
        const int i = b + lane;
        const uint32_t key = i < i1 ? keys[i] : 0u;
        const bool is_above = i < i1 && key > last, is_equal = i < i1 && key == last;
        const uint32_t ma = __ballot_sync(0xffffffffu, is_above), me = __ballot_sync(0xffffffffu, is_equal);
        const uint32_t na = xa + __popc(ma & below), ne = xe + __popc(me & below);
        if (is_above || (is_equal && ne < left)) out[a.sink + na + min(ne, left)] = a.sink + c0 + i;
        xa += __popc(ma);
        xe += __popc(me);
    }
    if (ranks > 1) {  // nobody leaves while another may still read its sums
        cluster_arrive();
        cluster_wait();
    }
}

template <int D, int NT>
static pa_status launch_select(const SelectArgs &a, int num_rows, cudaStream_t stream) {
    // enough CTAs to fill the machine, and no more than the pages can use
    const int64_t rows = static_cast<int64_t>(num_rows) * a.num_kv_heads;
    int ranks = 1;
    while (ranks < 8 && rows * ranks < 2 * 152 && a.max_blocks > 128 * ranks) ranks *= 2;
    while (ranks < 8 && a.max_blocks > 32768 * ranks) ranks *= 2;
    const size_t smem = static_cast<size_t>(((a.max_blocks + ranks - 1) / ranks + 15) & ~15) * 4;
    auto kern = select_kernel<D, NT>;
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
    if (head_dim == 128)
        return a.group <= 8 ? launch_select<128, 1>(a, num_rows, stream) : launch_select<128, 2>(a, num_rows, stream);
    return a.group <= 8 ? launch_select<64, 1>(a, num_rows, stream) : launch_select<64, 2>(a, num_rows, stream);
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
