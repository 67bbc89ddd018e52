// The int8 form that pages' bounds and queries are compared in, and the choice
// of a row's pages by a cluster of CTAs: shared by the kernel that only chooses
// and the one that goes on to attend.
#pragma once

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
    int stages;  // of the warps' rings of copies: 2 or 3
    unsigned int *err;
};

// Arguments checked by the caller (`err` may come out null: no CUDA device).
SelectArgs select_args(const void *q, const int8_t *summary, const int8_t *exponents, const int32_t *block_tables,
                       int max_blocks, const int32_t *context_lens, int num_q_heads, int num_kv_heads, int num_blocks,
                       int block_size, int top_k, int sink, int recent, int32_t *selected, int32_t *counts);
pa_status run_select(const SelectArgs &a, int num_rows, int head_dim, cudaStream_t stream);

// fp32 -> unsigned with the same order
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

// Four signed bytes of a word as fp16 pairs, even = bytes 0 and 2, odd = bytes
// 1 and 3: 0x6400 | (x + 128) is the fp16 value kOffset + x, exactly.
constexpr float kOffset = 1152.f;
__device__ __forceinline__ void int8x4_offset_f16(uint32_t w, uint32_t &even, uint32_t &odd) {
    even = (w & 0x00ff00ffu) ^ 0x64806480u;
    odd = ((w >> 8) & 0x00ff00ffu) ^ 0x64806480u;
}
__device__ __forceinline__ void int8x4_f16(uint32_t w, uint32_t &even, uint32_t &odd) {
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    int8x4_offset_f16(w, even, odd);
    const __half2 e = __hsub2(*reinterpret_cast<const __half2 *>(&even), off);
    const __half2 o = __hsub2(*reinterpret_cast<const __half2 *>(&odd), off);
    even = *reinterpret_cast<const uint32_t *>(&e);
    odd = *reinterpret_cast<const uint32_t *>(&o);
}

// stands in for the exponent of a page outside the pool: its score is -infinity
constexpr int kBadExp = -128;

// Shared memory of the choice, beside its keys and copies in flight.
template <int D, int NT, int kSelThreads>
struct alignas(16) Choice {
    static constexpr int kWarps = kSelThreads / 32;
    static constexpr int kBins = 4 * kSelThreads;  // of a histogram: four to a thread
    static constexpr int kBinBits = kSelThreads == 256 ? 10 : 9;
    static constexpr int kListMax = kSelThreads;   // keys that are ranked one against another
    static_assert((1 << kBinBits) == kBins, "bins");
    uint32_t hist[2][kBins];
    int8_t query[8 * NT][2 * D];  // the group's queries as whole numbers
    float unit[8 * NT];           // what they are whole numbers of
    float sum[8 * NT][D / 64];    // and their sums over 64 dims
    uint32_t list[kListMax], ranked[kListMax];
    uint32_t list_len;
    uint32_t range[2];  // least and largest key of the CTA
    uint32_t warp_sum[2][kWarps];
    uint32_t pick[3];
    uint32_t taken[2];  // pages above, and equal to, the last key
    uint32_t bits[16];  // pages taken, of few
};

// Up to this many candidates, no more than one to a thread, are ranked one
// against another with no histogram, which costs a cluster five barriers (8 rows
// of 313 pages, 8 CTAs each, choice and attention: 14.3 us with it, 12.4 without;
// but 17 with half a thousand keys for each thread to look at).
constexpr int kFew = 500;

// What a row attends to: `count` logical pages, listed, or the first ones when
// `list` is null.
struct Chosen {
    int count;
    const int32_t *list;
};

// A warp takes 16 pages' bounds at a time through a ring of `stages` such steps
// of its own.
constexpr int kStepPages = 16;
constexpr int kMaxStages = 3;
__host__ __device__ constexpr int copy_bytes(int threads, int head_dim, int stages) {
    return threads / 32 * stages * kStepPages * 2 * head_dim;
}
// Bytes of keys that a CTA needs when `ranks` share a row.
inline int key_bytes(int max_blocks, int ranks) { return ((((max_blocks + ranks - 1) / ranks + 31) & ~31) + 4) * 4; }

// The cluster's choice for row t and KV head h, written to a.selected and
// a.counts, and returned.
//
// Scores: 16 pages x 8 query heads x 16 bounds are one m16n8k16 product in
// fp16, which every int8 value is, with fp32 sums.  A lane takes 16-byte pieces
// of a page's bounds and of a query; the order of the sum is free, so both
// sides take the order that the bytes lie in.  A bound becomes fp16 as 1152 + x
// (three instructions for four of them) and the sums start at -1152 times the
// query's, so they come out as they should; over 64 head dims they stay below
// 64 * 127 * (1152 + 127) < 2^24, where fp32 holds every whole number.  (The
// product of signed bytes needs no conversion, but takes 16 cycles an SM for
// twice the depth of this one's 2: with 16 query heads it measured 51 against
// 40 us over 8 rows of 8192 pages.)
// Choice: a histogram of the keys over their own range, the bin that holds the
// last page to be taken, and, once few keys are left in the bin, their ranks
// among one another; of few candidates, their ranks at once.
//
// `copies` is copy_bytes() of shared memory (16-byte aligned), `keys`
// key_bytes().  Every thread of the cluster calls it; on return the listed pages
// are visible to all of them.
template <int D, int NT, int kSelThreads>
__device__ __forceinline__ Chosen choose(const SelectArgs &a, uint8_t *copies, uint32_t *keys, Choice<D, NT, kSelThreads> &sh,
                                         int rank, int ranks, int h, int t) {
    using S = Choice<D, NT, kSelThreads>;
    constexpr int kSelWarps = S::kWarps, kBins = S::kBins, kBinBits = S::kBinBits, kListMax = S::kListMax;
    constexpr int PIECES = 2 * D / 64;  // 16-byte pieces of a page that a lane reads
    constexpr int SETS = D / 64;        // accumulators of a product, 64 head dims each
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

    // the group's queries, eight dims a thread
    constexpr int TPH = D / 8;  // threads to a head
    constexpr int QV = (8 * NT * TPH + kSelThreads - 1) / kSelThreads;
    uint4 qraw[QV];
#pragma unroll
    for (int i = 0; i < QV; ++i) {
        const int g = min((i * kSelThreads + tid) / TPH, a.group - 1);
        qraw[i] = *(reinterpret_cast<const uint4 *>(a.q + (out_row * a.group + g) * D) + tid % TPH);
    }
    // with one CTA to the row its first pages are known before the length is
    const int32_t *table = a.block_tables + static_cast<int64_t>(t) * a.max_blocks + a.sink;
    int32_t next_blk = -1;
    {
        const int at = warp * kStepPages + lane % kStepPages;
        if (ranks == 1 && a.sink + at < a.max_blocks) next_blk = table[at];
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
        return Chosen{count, nullptr};
    }
    const int want = a.top_k - a.sink - a.recent;  // pages to take from the candidates
    for (int i = rank * kSelThreads + tid; i < a.sink; i += ranks * kSelThreads) out[i] = i;
    for (int i = rank * kSelThreads + tid; i < a.recent; i += ranks * kSelThreads)
        out[a.top_k - a.recent + i] = nb - a.recent + i;
    if (want == 0) {
        sync_all();
        return Chosen{count, out};
    }

    const int ncand = nb - a.sink - a.recent;
    const int per = ((ncand + ranks - 1) / ranks + 31) & ~31;
    const int c0 = min(ncand, rank * per), c1 = min(ncand, c0 + per);
    const int have = c1 - c0;
    const bool few = per <= kSelThreads && ncand <= kFew && a.top_k <= kBins;
    // The warp's i-th step is pages (i * warps + warp) * STEP and on of the
    // share.  Their bounds are copied 16 bytes a lane, stages - 1 steps ahead;
    // piece x of page p lies at x ^ 4 (p & 1), so that eight lanes' reads below
    // meet eight bank groups.
    constexpr int PAGE = 2 * D;
    constexpr int STEP = kStepPages;
    constexpr int LPP = PAGE / 16;     // lanes to a page
    constexpr int PPC = 32 / LPP;      // pages per copy instruction
    const int own = lane % STEP;       // the step's page that the lane looks up
    const int steps = have > warp * STEP ? (have - warp * STEP + STEP * kSelWarps - 1) / (STEP * kSelWarps) : 0;
    if (ranks > 1 && warp * STEP + own < have) next_blk = table[c0 + warp * STEP + own];
    const uint8_t *ring = copies + warp * a.stages * STEP * PAGE;
    const uint32_t ring_at = smem_addr(ring);
    int put = 0;
    int exps0 = 0, exps1 = 0, exps2 = 0;  // exponents of the lane's pages, by age
    auto copy = [&](int i) {
        exps2 = exps1;
        exps1 = exps0;
        if (i < steps) {
            const int at = (i * kSelWarps + warp) * STEP + own;
            int32_t blk = next_blk;
            next_blk = at + STEP * kSelWarps < have ? table[c0 + at + STEP * kSelWarps] : -1;
            const bool bad = blk < 0 || blk >= a.num_blocks;
            if (bad) {
                if (at < have) set_device_error(a.err, PA_DEVERR_BAD_BLOCK);
                blk = 0;
            }
            const int32_t row = blk * a.num_kv_heads + h;  // below 2^27: the pool's limit
            const uint32_t dst = ring_at + put * STEP * PAGE;
            put = put + 1 == a.stages ? 0 : put + 1;
#pragma unroll
            for (int k = 0; k < STEP; k += PPC) {
                const int p = k + lane / LPP, x = lane % LPP;
                const int32_t prow = __shfl_sync(0xffffffffu, row, p);
                cp_async16(dst + p * PAGE + ((x ^ ((p & 1) << 2)) << 4),
                           a.summary + static_cast<int64_t>(prow) * PAGE + x * 16);
            }
            exps0 = bad ? kBadExp : a.exponents[row];
        }
        cp_async_commit();
    };
    if (tid == 0) {
        sh.range[0] = 0xffffffffu;
        sh.range[1] = 0;
        sh.list_len = 0;
    }
    if (!few) {
#pragma unroll
        for (int i = 0; i < 2; ++i) reinterpret_cast<uint4 *>(sh.hist[i])[tid] = make_uint4(0, 0, 0, 0);
    } else if (ranks > 1) {
        cluster_arrive();  // the others may write to this CTA's shared memory
    }

    // queries as whole numbers: their positive parts (for the largest keys),
    // then the negative ones (for the least)
#pragma unroll
    for (int i = 0; i < QV; ++i) {
        const int v = i * kSelThreads + tid, g = v / TPH;
        const uint32_t w[4] = {qraw[i].x, qraw[i].y, qraw[i].z, qraw[i].w};
        float x[8], amax = 0.f;
        bool odd = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[j]));
            x[2 * j] = f.x;
            x[2 * j + 1] = f.y;
            odd |= !(fabsf(f.x) < INFINITY) || !(fabsf(f.y) < INFINITY);
            amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
        const uint32_t votes = __ballot_sync(0xffffffffu, odd);
        odd = (votes >> (lane & ~(TPH - 1))) & ((1u << TPH) - 1u);
#pragma unroll
        for (int m = 1; m < TPH; m <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
        const int e = odd ? kMinExp : shared_exponent(amax);
        const float inv = power_of_two(-e);
        uint32_t pos[2] = {0, 0}, neg[2] = {0, 0};
        int total = 0;  // of 64 dims
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int y = odd ? 0 : to_int8(x[j], inv);
            total += y;
            pos[j / 4] |= static_cast<uint32_t>(max(y, 0)) << (8 * (j % 4));
            neg[j / 4] |= (static_cast<uint32_t>(min(y, 0)) & 0xffu) << (8 * (j % 4));
        }
#pragma unroll
        for (int m = 1; m < 8; m <<= 1) total += __shfl_xor_sync(0xffffffffu, total, m);
        if (g < 8 * NT) {
            reinterpret_cast<uint2 *>(sh.query[g])[tid % TPH] = make_uint2(pos[0], pos[1]);
            reinterpret_cast<uint2 *>(sh.query[g])[TPH + tid % TPH] = make_uint2(neg[0], neg[1]);
            if (tid % TPH == 0) sh.unit[g] = power_of_two(e);
            if (tid % 8 == 0) sh.sum[g][tid % TPH / 8] = static_cast<float>(total);
        }
    }
    for (int i = 0; i < a.stages - 1; ++i) copy(i);
    __syncthreads();
    // B fragments: lane (r, c) holds pieces c, c + 4, ... of head r
    uint32_t qf[NT][PIECES][4][2];
    float unit[NT][2], start[NT][SETS][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const uint4 w = reinterpret_cast<const uint4 *>(sh.query[nt * 8 + r])[c + 4 * i];
            int8x4_f16(w.x, qf[nt][i][0][0], qf[nt][i][0][1]);
            int8x4_f16(w.y, qf[nt][i][1][0], qf[nt][i][1][1]);
            int8x4_f16(w.z, qf[nt][i][2][0], qf[nt][i][2][1]);
            int8x4_f16(w.w, qf[nt][i][3][0], qf[nt][i][3][1]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            unit[nt][j] = sh.unit[nt * 8 + 2 * c + j];
#pragma unroll
            for (int k = 0; k < SETS; ++k) start[nt][k][j] = -kOffset * sh.sum[nt * 8 + 2 * c + j][k];
        }
    }

    // ---- scores of this CTA's share of the candidates -------------------------
    if (few && ranks > 1) cluster_wait();
    uint32_t kmin = 0xffffffffu, kmax = 0;
    int get = 0;
    for (int it = 0; it < steps; ++it) {
        copy(it + a.stages - 1);
        if (a.stages == 3)
            cp_async_wait<2>();
        else
            cp_async_wait<1>();
        __syncwarp();
        const int exps = a.stages == 3 ? exps2 : exps1;
        const uint8_t *stage = ring + get * STEP * PAGE;
        get = get + 1 == a.stages ? 0 : get + 1;
        // each 64 head dims have sums of their own: two chains of eight products
        float acc[NT][SETS][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < SETS; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nt][k][e] = start[nt][k][e & 1];
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int x = ((c + 4 * i) ^ ((r & 1) << 2)) << 4;
            const uint4 w0 = *reinterpret_cast<const uint4 *>(stage + r * PAGE + x);
            const uint4 w1 = *reinterpret_cast<const uint4 *>(stage + (r + 8) * PAGE + x);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                auto word = [&](const uint4 &u) { return j == 0 ? u.x : j == 1 ? u.y : j == 2 ? u.z : u.w; };
                uint32_t a0, a1, a2, a3;
                int8x4_offset_f16(word(w0), a0, a2);
                int8x4_offset_f16(word(w1), a1, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma16816<true>(acc[nt][i % SETS], a0, a1, a2, a3, qf[nt][i][j][0], qf[nt][i][j][1]);
            }
        }
        auto dot = [&](int nt, int e) {
            float x = acc[nt][0][e];
            if constexpr (SETS == 2) x += acc[nt][1][e];
            return x;
        };
        float s0 = -INFINITY, s1 = -INFINITY;  // pages r and r + 8
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (nt * 8 + 2 * c + j < a.group) {
                    s0 = fmaxf(s0, dot(nt, j) * unit[nt][j]);
                    s1 = fmaxf(s1, dot(nt, 2 + j) * unit[nt][j]);
                }
#pragma unroll
        for (int m = 1; m < 4; m <<= 1) {
            s0 = fmaxf(s0, __shfl_xor_sync(0xffffffffu, s0, m));
            s1 = fmaxf(s1, __shfl_xor_sync(0xffffffffu, s1, m));
        }
        const int page = r + 8 * (c & 1);
        const int ex = __shfl_sync(0xffffffffu, exps, page);
        const int i = (it * kSelWarps + warp) * STEP + page;  // of the CTA's share
        if (c < 2 && i < have) {
            const float score = ex == kBadExp ? -INFINITY : ex == kOddExp ? INFINITY : (c ? s1 : s0) * power_of_two(ex);
            const uint32_t key = order_key(score + 0.f);  // no negative zero
            keys[i] = key;
            if (few && ranks > 1)
                for (int k = 0; k < ranks; ++k) st_cluster_u32(smem_addr(&sh.hist[0][c0 + i]), k, key);
            kmin = min(kmin, key);
            kmax = max(kmax, key);
        }
        __syncwarp();  // the step's place in the ring is free
    }
    if (few) {
        // Every CTA has all keys (its own, or every CTA's in sh.hist[0]) and
        // ranks its own pages among them: one is taken when fewer than `want`
        // come before it, by key and then by index.  The bits that say which
        // were taken go to every CTA.
        uint32_t *all = ranks > 1 ? sh.hist[0] : keys;
        if (tid < 3) all[ncand + tid] = 0u;  // to a multiple of four, below every score's key
        sh.ranked[tid] = 0;
        sync_all();
        // `split` threads to a page, each with its part of the keys
        const int split = have <= kSelThreads / 4 ? 4 : have <= kSelThreads / 2 ? 2 : 1;
        const int mine = tid % (kSelThreads / split), part = tid / (kSelThreads / split);
        const int self = c0 + mine;
        if (mine < have) {
            const uint32_t key = all[self];
            uint32_t place = 0;
#pragma unroll 4
            for (int j = 4 * part; j < ncand; j += 4 * split) {
                const uint4 k4 = *reinterpret_cast<const uint4 *>(all + j);
                place += k4.x > key || (k4.x == key && j < self);
                place += k4.y > key || (k4.y == key && j + 1 < self);
                place += k4.z > key || (k4.z == key && j + 2 < self);
                place += k4.w > key || (k4.w == key && j + 3 < self);
            }
            if (split > 1) atomicAdd(&sh.ranked[mine], place);
            else sh.ranked[mine] = place;
        }
        __syncthreads();
        if (warp * 32 < have) {
            const bool is = warp * 32 + lane < have && sh.ranked[warp * 32 + lane] < static_cast<uint32_t>(want);
            const uint32_t votes = __ballot_sync(0xffffffffu, is);
            if (lane < ranks) {
                if (ranks > 1)
                    st_cluster_u32(smem_addr(&sh.bits[c0 / 32 + warp]), lane, votes);
                else
                    sh.bits[warp] = votes;
            }
        }
        sync_all();
        // each page's place in the list: those taken in the words before its own
        int32_t *list = reinterpret_cast<int32_t *>(sh.hist[1]);
        const int words = (ncand + 31) / 32;
        const int in_word = lane < words ? __popc(sh.bits[lane]) : 0;
        int upto = in_word;
#pragma unroll
        for (int m = 1; m < 16; m <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, upto, m);
            if (lane >= m) upto += o;
        }
        for (int w = warp; w < words; w += kSelWarps) {
            const uint32_t word = sh.bits[w];
            const int before = __shfl_sync(0xffffffffu, upto - in_word, w);
            if (word >> lane & 1u) {
                const int at = a.sink + before + __popc(word & ((1u << lane) - 1u));
                const int page = a.sink + 32 * w + lane;
                list[at] = page;
                if (rank == 0) out[at] = page;
            }
        }
        for (int i = tid; i < a.sink; i += kSelThreads) list[i] = i;
        for (int i = tid; i < a.recent; i += kSelThreads) list[a.top_k - a.recent + i] = nb - a.recent + i;
        __syncthreads();
        return Chosen{count, list};
    }
    // four keys behind the share: 0, below every score's
    if (tid < 4) keys[have + tid] = 0u;
    kmin = __reduce_min_sync(0xffffffffu, kmin);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    if (lane == 0) {
        atomicMin(&sh.range[0], kmin);
        atomicMax(&sh.range[1], kmax);
    }
    sync_all();

    // ---- the key of the last page taken ---------------------------------------
    uint32_t low = sh.range[0], high = sh.range[1];
    if (ranks > 1) {  // a lane for each CTA
        low = __reduce_min_sync(0xffffffffu, lane < ranks ? ld_cluster_u32(smem_addr(&sh.range[0]), lane) : 0xffffffffu);
        high = __reduce_max_sync(0xffffffffu, lane < ranks ? ld_cluster_u32(smem_addr(&sh.range[1]), lane) : 0u);
    }
    uint32_t span = high - low;  // keys looked at: low .. low + span
    int shift = max(0, 32 - __clz(span) - kBinBits);
    uint32_t left = want;  // pages still to be found among them
    uint32_t last;         // the last key taken, by the `left` first pages that have it
    for (int pass = 0;; ++pass) {
        uint32_t *hs = sh.hist[pass & 1];
        for (int i = 4 * tid; i < have; i += 4 * kSelThreads) {
            const uint4 k4 = *reinterpret_cast<const uint4 *>(keys + i);
            const uint32_t d[4] = {k4.x - low, k4.y - low, k4.z - low, k4.w - low};  // of a key below: past span
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (d[k] <= span) atomicAdd(&hs[d[k] >> shift], 1u);
        }
        sync_all();
        // four bins to a thread, from the top
        const uint32_t at = smem_addr(hs) + (kSelThreads - 1 - tid) * 16;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (ranks > 1) {
            uint4 o[8];  // all in flight together
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = k < ranks ? ld_cluster_v4(at, k) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v.x += o[k].x;
                v.y += o[k].y;
                v.z += o[k].z;
                v.w += o[k].w;
            }
        } else {
            v = lds128(at);
        }
        const uint32_t sum = v.x + v.y + v.z + v.w;
        uint32_t before = sum;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, before, m);
            if (lane >= m) before += o;
        }
        if (lane == 31) sh.warp_sum[0][warp] = before;
        before -= sum;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kSelWarps; ++w)
            if (w < warp) before += sh.warp_sum[0][w];
        if (before < left && before + sum >= left) {
            const uint32_t bins[4] = {v.w, v.z, v.y, v.x};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (before < left && before + bins[k] >= left) {
                    sh.pick[0] = kBins - 1 - (4 * tid + k);
                    sh.pick[1] = left - before;
                    sh.pick[2] = bins[k];
                }
                before += bins[k];
            }
        }
        // the histogram of the pass before: every CTA has read it
        if (pass > 0) reinterpret_cast<uint4 *>(sh.hist[(pass + 1) & 1])[tid] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        low += sh.pick[0] << shift;
        left = sh.pick[1];
        const uint32_t found = sh.pick[2];
        span = (1u << shift) - 1u;
        if (found <= kListMax) {
            // the bin's keys, gathered in the first CTA, ranked by every CTA
            for (int i = 4 * tid; i < have; i += 4 * kSelThreads) {
                const uint4 k4 = *reinterpret_cast<const uint4 *>(keys + i);
                const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (k[u] - low <= span) {
                        if (ranks > 1)
                            st_cluster_u32(smem_addr(sh.list) + 4 * atom_add_cluster(smem_addr(&sh.list_len), 0, 1u), 0, k[u]);
                        else
                            sh.list[atomicAdd(&sh.list_len, 1u)] = k[u];
                    }
            }
            sync_all();
            const uint32_t key = tid >= found ? 0u : ranks > 1 ? ld_cluster_u32(smem_addr(sh.list) + 4 * tid, 0) : sh.list[tid];
            sh.ranked[tid] = key;
            __syncthreads();
            uint32_t greater = 0, equal = 0;
            for (uint32_t j = 0; j < found; ++j) {
                greater += sh.ranked[j] > key;
                equal += sh.ranked[j] == key;
            }
            if (tid < found && greater < left && greater + equal >= left) {
                sh.pick[0] = key;  // by every page that has it: the same values
                sh.pick[1] = left - greater;
            }
            __syncthreads();
            last = sh.pick[0];
            left = sh.pick[1];
            break;
        }
        if (shift == 0) {  // one key, more often than the list is long
            last = low;
            break;
        }
        shift = max(0, shift - kBinBits);
    }

    // ---- every key above `last`, and the first `left` equal to it --------------
    // a warp takes a run of pages, a lane four in a row
    const int seg = ((have + kSelWarps - 1) / kSelWarps + 127) & ~127;
    const int i0 = min(have, warp * seg), i1 = min(have, i0 + seg);
    // of the four keys from i on: above | equal << 16, and a bit for each
    auto look = [&](int i, uint32_t &ma, uint32_t &me) -> uint32_t {
        ma = me = 0;
        if (i < i1) {
            const uint4 k4 = *reinterpret_cast<const uint4 *>(keys + i);
            const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                ma |= (k[u] > last ? 1u : 0u) << u;
                me |= (k[u] == last ? 1u : 0u) << u;
            }
        }
        return __popc(ma) | __popc(me) << 16;
    };
    uint32_t above = 0, equal = 0;
    for (int i = i0 + 4 * lane; i < i1; i += 128) {
        uint32_t ma, me;
        look(i, ma, me);
        above += __popc(ma);
        equal += __popc(me);
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
        sh.warp_sum[0][warp] = above;
        sh.warp_sum[1][warp] = equal;
    }
    __syncthreads();
    uint32_t xa = 0, xe = 0;  // taken, and equal, before this warp's
    if (ranks > 1) {
        if (tid == 0) {
            uint32_t sa = 0, se = 0;
            for (int w = 0; w < kSelWarps; ++w) {
                sa += sh.warp_sum[0][w];
                se += sh.warp_sum[1][w];
            }
            sh.taken[0] = sa;
            sh.taken[1] = se;
        }
        sync_all();
        xa = __reduce_add_sync(0xffffffffu, lane < rank ? ld_cluster_u32(smem_addr(&sh.taken[0]), lane) : 0u);
        xe = __reduce_add_sync(0xffffffffu, lane < rank ? ld_cluster_u32(smem_addr(&sh.taken[1]), lane) : 0u);
    }
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w)
        if (w < warp) {
            xa += sh.warp_sum[0][w];
            xe += sh.warp_sum[1][w];
        }
    for (int b = i0; b < i1; b += 128) {
        const int i = b + 4 * lane;
        uint32_t ma, me;
        const uint32_t own = look(i, ma, me);
        uint32_t upto = own;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, upto, m);
            if (lane >= m) upto += o;
        }
        uint32_t na = xa + ((upto - own) & 0xffffu), ne = xe + ((upto - own) >> 16);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const bool is_above = ma >> u & 1, is_equal = me >> u & 1;
            if (is_above || (is_equal && ne < left)) out[a.sink + na + min(ne, left)] = a.sink + c0 + i + u;
            na += is_above;
            ne += is_equal;
        }
        const uint32_t all = __shfl_sync(0xffffffffu, upto, 31);
        xa += all & 0xffffu;
        xe += all >> 16;
    }
    sync_all();  // the list is complete, and nobody leaves while another may still read its sums
    return Chosen{count, out};
}

}  // namespace sparse
}  // namespace pa
