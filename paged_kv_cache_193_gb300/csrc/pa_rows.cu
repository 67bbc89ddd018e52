// Attention of many query rows to one run of cached pages (pa_rows.cuh) on the
// tcgen05 tensor cores.
//
// One CTA to (two neighbouring tiles of 128 rows, part of the keys, KV head,
// sequence or group).  A run's keys go by in blocks of 64 through a ring of
// stages that both tiles read.  Per tile and block:
//   S = Q K^T  (M 128, N 64, K head dim) into one of two buffers in tensor
//              memory, both operands K-major from shared memory;
//   softmax    a row (lane of tensor memory) to a thread, no exchange between
//              threads: the block's largest score, probabilities against a
//              reference that moves only when a row outgrows it by 2^8, written
//              over S as 16-bit pairs;
//   O += P V   (M 128, N head dim, K 64), P from tensor memory, V as it lies in
//              its pages.
// S(j + 1) is made while the softmax works on S(j).
//
// Warps: 0-3 and 4-7 the tiles' softmax, 8 and 10 the copies of K and V pages
// (2-D TMA, a lane to a page), 9 and 11 the tiles' products.  With an E4M3
// cache the pages land in a ring of their own, and warps 12-15 widen them to
// fp16 (exact), a row of K or V to a thread, in the layout that bf16 pages land
// in.  A part's keys from the run's end on are masked, and V's rows there are
// zeros: behind the end lies anything, and 0 times that could be NaN.
//
// Every wait is bounded (2 s unless a test sets another limit).
#include <cudaTypedefs.h>
#include <limits.h>
#include <math.h>

#include <atomic>

#include "pa_prefill.cuh"
#include "pa_rows.cuh"
#include "pa_sparse.cuh"

namespace pa {

namespace rows {

constexpr int kLoadK = 8, kLoadV = 10, kMma0 = 9, kMma1 = 11, kWiden = 12;  // warps
constexpr int kQSlab = kRows * 128;   // 64 dims of a tile's queries
constexpr int kKVSlab = kKeys * 128;  // 64 dims of a block's keys or values
constexpr int kTmemCols = 512;        // a tile: S at 0 and 64, O at 128
constexpr int kOCol = 128;
constexpr float kLazy = 8.f;
// fp16 probabilities are taken times 2^7: up to 2^15 against the reference's
// 2^8, and whole bits down to 2^-21.
constexpr float kRaise = 128.f;
constexpr uint64_t kDrainNs = 2000000000ull;

template <int D, bool FP8>
struct Layout {
    static constexpr int kThreads = FP8 ? 512 : 384;
    static constexpr int kSlabs = D / 64;
    static constexpr int kQTile = kSlabs * kQSlab;
    static constexpr int kStage = kSlabs * kKVSlab;  // a block of K, or of V, as 16-bit rows
    static constexpr int kStages = (FP8 ? 3 : 5) * 2 / kSlabs;
    static constexpr int kRaw = kKeys * D;  // a block of E4M3 K, or V
    static constexpr int kRawStages = FP8 ? 4 * 2 / kSlabs : 0;
    static constexpr int kK = kTiles * kQTile;
    static constexpr int kV = kK + kStages * kStage;
    static constexpr int kRawK = kV + kStages * kStage;
    static constexpr int kRawV = kRawK + kRawStages * kRaw;
    static constexpr int kSmem = kRawV + kRawStages * kRaw + 1024;
};

// Which rows and which keys a CTA has.
struct Work {
    int token0;  // first token of the rows that the pair's sequence or group has
    int tokens;  // how many it has
    int at;      // the pair's first of them
    int table;   // whose table row leads to the keys
    int keys;    // of the whole run
    int part;
};

// Called by whole warps; every warp comes to the same answer.  False: nothing to do.
__device__ __forceinline__ bool find_work(const Args &a, Work &w) {
    const int lane = threadIdx.x & 31;
    const int cap = a.max_blocks * a.block_size;
    int pair = blockIdx.x / a.parts;
    w.part = blockIdx.x - pair * a.parts;
    if (!a.group_start) {
        const int s = blockIdx.z;
        const bool good = query_range(a, s, w.token0, w.tokens);
        w.at = kTiles * pair * a.tile_tokens;
        w.table = s;
        w.keys = max(a.lens[s], 0);
        if (!good || w.keys > cap) {
            if (threadIdx.x == 0) set_device_error(a.err, PA_DEVERR_BAD_CONTEXT);
            w.keys = min(w.keys, cap);
        }
        return good && w.at < w.tokens;
    }
    // The pair's group: the groups' pairs lie one after the other.
    int first = 0, end = 0, pages = 0;
    bool found = false;
    for (int g0 = 0; g0 < a.num_groups && !found; g0 += 32) {
        const int g = g0 + lane;
        int lo = 0, hi = 0, n = 0;
        if (g < a.num_groups) {
            lo = min(max(a.group_start[g], 0), a.num_seqs);
            hi = min(max(a.group_start[g + 1], lo), a.num_seqs);
            n = min(max(a.prefix_blocks[g], 0), a.max_prefix_blocks);
        }
        const int mine = (hi - lo + kTiles * a.tile_tokens - 1) / (kTiles * a.tile_tokens);
        int before = mine;  // sum of the lanes' up to and with this one
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int x = __shfl_up_sync(0xffffffffu, before, d);
            if (lane >= d) before += x;
        }
        const unsigned has = __ballot_sync(0xffffffffu, before > pair);
        found = has != 0;
        const int pick = found ? __ffs(has) - 1 : 31;
        const int behind = __shfl_sync(0xffffffffu, before, pick);
        if (found) {
            pair -= behind - __shfl_sync(0xffffffffu, mine, pick);
            first = __shfl_sync(0xffffffffu, lo, pick);
            end = __shfl_sync(0xffffffffu, hi, pick);
            pages = __shfl_sync(0xffffffffu, n, pick);
        } else {
            pair -= behind;
        }
    }
    if (!found || pages == 0) return false;
    w.token0 = first;
    w.tokens = end - first;
    w.at = kTiles * pair * a.tile_tokens;
    w.keys = pages * a.block_size;
    // The table row of the pair's first sequence that has the whole prefix; the
    // others have none of it to themselves, and their rows here are not read.
    const int s0 = first + w.at, s1 = min(end, s0 + kTiles * a.tile_tokens);
    w.table = -1;
    for (int s = s0; s < s1 && w.table < 0; s += 32) {
        const int len = s + lane < s1 ? a.lens[s + lane] : 0;
        const unsigned has = __ballot_sync(0xffffffffu, len >= w.keys);
        if (has) w.table = s + __ffs(has) - 1;
    }
    return w.table >= 0;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(Layout<D, FP8>::kThreads, 1)
    rows_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const Args a) {
    using L = Layout<D, FP8>;
    constexpr int kStages = L::kStages, kRawStages = FP8 ? L::kRawStages : 1;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t q_full, v_zeroed, stall_bar;
    // a stage's K and V are in place (kv_full); both tiles' products have read it (kv_empty)
    __shared__ __align__(8) uint64_t kv_full[kStages], kv_empty[kStages];
    // E4M3 K (0) and V (1) pages have landed, have been read; a tile's queries are fp16
    __shared__ __align__(8) uint64_t raw_full[2][kRawStages], raw_empty[2][kRawStages], q_conv[kTiles];
    // per tile: S(j) is in buffer j % 2, P(j) is over it, PV(j) is done, all is done
    __shared__ __align__(8) uint64_t s_full[kTiles][2], p_full[kTiles][2], pv_done[kTiles], drain[kTiles];
    __shared__ uint32_t tmem_base_s;
    __shared__ int failed_s;

    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint64_t limit = a.wait_limit_ns;
    const int h = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    dependent_wait();
    // The kernel that reads a prefix's parts begins with work that needs none of
    // them, and waits for this one's end itself.
    if (a.group_start) dependent_release();
    Work w;
    if (!find_work(a, w)) return;
    const int all = (w.keys + kKeys - 1) / kKeys, each = blocks_per_part(all, a.parts);
    const int first = w.part * each, nkb = min(each, all - first);  // this part's blocks
    const int ntiles = w.at + a.tile_tokens < w.tokens ? 2 : 1;
    auto tokens_of = [&](int T) { return min(a.tile_tokens, w.tokens - w.at - T * a.tile_tokens); };
    auto warps_of = [&](int T) { return (tokens_of(T) * a.group + 31) / 32; };  // with a live row
    if (nkb <= 0) {
        if (a.out && w.keys == 0) {  // nothing to attend to
            const int n = min(w.tokens - w.at, kTiles * a.tile_tokens) * a.group * (D / 8);
            for (int i = tid; i < n; i += L::kThreads) {
                const int row = i / (D / 8), t = row / a.group;
                __nv_bfloat16 *to = a.out + ((static_cast<int64_t>(w.token0) + w.at + t) * a.num_q_heads + h * a.group + row % a.group) * D;
                *reinterpret_cast<uint4 *>(to + i % (D / 8) * 8) = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        return;
    }
    const int left = w.keys - first * kKeys;           // of the run, from this part's first key on
    const bool partial = left < nkb * kKeys;           // the last block reaches behind the run's end

    // A loader's lane has a page of every block; its table entry is read a block ahead.
    const int pages = kKeys / a.block_size;
    const int32_t *table = a.block_tables + static_cast<int64_t>(w.table) * a.max_blocks;
    constexpr int kBehind = INT_MIN;
    auto page_entry = [&](int kb) {
        const int page = (first + kb) * pages + lane;
        return lane < pages && page * a.block_size < w.keys ? table[page] : kBehind;
    };
    const bool loader = warp == kLoadK || warp == kLoadV;
    const int e_first = loader ? page_entry(0) : kBehind;

    if (tid == 0) {
        mbar_init(smem_addr(&q_full), 1);
        mbar_init(smem_addr(&v_zeroed), 1);
        mbar_init(smem_addr(&stall_bar), 1);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_addr(&kv_full[i]), FP8 ? 4 : 2);  // the widening warps, or the loaders
            mbar_init(smem_addr(&kv_empty[i]), ntiles);
        }
        if constexpr (FP8)
            for (int i = 0; i < 2 * kRawStages; ++i) {
                mbar_init(smem_addr(&raw_full[i & 1][i >> 1]), 1);
                mbar_init(smem_addr(&raw_empty[i & 1][i >> 1]), 2);
            }
        for (int t = 0; t < ntiles; ++t) {
            for (int b = 0; b < 2; ++b) {
                mbar_init(smem_addr(&s_full[t][b]), 1);
                mbar_init(smem_addr(&p_full[t][b]), warps_of(t));
            }
            mbar_init(smem_addr(&pv_done[t]), 1);
            mbar_init(smem_addr(&drain[t]), 1);
            mbar_init(smem_addr(&q_conv[t]), warps_of(t));
        }
        failed_s = 0;
        fence_barrier_init();
        const int q_box = D * 2 * a.group * a.tile_tokens;
        mbar_arrive_expect_tx(smem_addr(&q_full), ntiles * q_box);
        for (int T = 0; T < ntiles; ++T)
            for (int sl = 0; sl < L::kSlabs; ++sl)
                tma_load_3d(base + T * L::kQTile + sl * kQSlab, &tmQ, sl * 64, h * a.group,
                            w.token0 + w.at + T * a.tile_tokens, smem_addr(&q_full));
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (warp == kMma0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_base_s)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    auto fail = [&]() {
        set_device_error(a.err, PA_DEVERR_TIMEOUT);
        atomicExch(&failed_s, 1);
    };
    // a whole warp waits
    auto wait = [&](uint64_t &bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait_suspend(smem_addr(&bar), parity, limit)) != 0;
    };

    if (loader) {
        // ---------------- copies of pages ----------------
        const bool is_k = warp == kLoadK;
        const int rows_total = a.num_blocks * a.num_kv_heads * a.block_size;
        const CUtensorMap *map = is_k ? &tmK : &tmV;
        const uint64_t policy = l2_evict_first_policy();
        constexpr int kRing = FP8 ? kRawStages : kStages;
        constexpr int kBytes = FP8 ? L::kRaw : L::kStage;
        const uint32_t ring = base + (FP8 ? (is_k ? L::kRawK : L::kRawV) : (is_k ? L::kK : L::kV));
        uint64_t *full = FP8 ? raw_full[is_k ? 0 : 1] : kv_full, *empty = FP8 ? raw_empty[is_k ? 0 : 1] : kv_empty;
        int entry = e_first;
        for (int kb = 0; kb < nkb; ++kb) {
            const int st = kb % kRing;
            // pages behind the run, and bad entries (which are reported), are rows
            // behind the tensor's end: the copy fills zeros
            int y = rows_total;
            if (entry >= 0 && entry < a.num_blocks)
                y = (entry * a.num_kv_heads + h) * a.block_size;
            else if (entry != kBehind)
                set_device_error(a.err, PA_DEVERR_BAD_BLOCK);
            if (kb + 1 < nkb) entry = page_entry(kb + 1);
            const bool freed = wait(empty[st], (kb / kRing & 1) ^ 1);
            if (lane == 0) {
                if (!freed) fail();
                mbar_arrive_expect_tx(smem_addr(&full[st]), kBytes);
            }
            __syncwarp();
            if (lane < pages) {
                if constexpr (FP8) {
                    tma_load_2d(ring + st * kBytes + lane * a.block_size * D, map, 0, y, smem_addr(&full[st]), policy);
                } else {
                    for (int sl = 0; sl < L::kSlabs; ++sl)
                        tma_load_2d(ring + st * kBytes + sl * kKVSlab + lane * a.block_size * 128, map, sl * 64, y,
                                    smem_addr(&full[st]), policy);
                }
            }
        }
        if (!FP8 && !is_k && partial) {
            const int kb = nkb - 1, st = kb % kStages;
            if (!wait(kv_full[st], kb / kStages & 1) && lane == 0) fail();
            for (int r = left - kb * kKeys + lane; r < kKeys; r += 32)
                for (int sl = 0; sl < L::kSlabs; ++sl)
                    for (int c = 0; c < 8; ++c) st_shared_zero16(ring + st * kBytes + sl * kKVSlab + r * 128 + c * 16);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&v_zeroed));
        }
        // whatever gave up, the CTA ends after its copies: those of the last blocks may be in flight
        if (lane == 0)
            for (int kb = max(0, nkb - kRing); kb < nkb; ++kb)
                mbar_wait_suspend(smem_addr(&full[kb % kRing]), kb / kRing & 1, kDrainNs);
    } else if (warp == kMma0 || warp == kMma1) {
        // ---------------- products ----------------
        const int T = warp == kMma0 ? 0 : 1;
        if (T < ntiles) {
            constexpr uint32_t idesc_qk = FP8 ? tc_idesc_f16(kRows, kKeys, 0, 0) : tc_idesc_bf16(kRows, kKeys, 0, 0);
            constexpr uint32_t idesc_pv = FP8 ? tc_idesc_f16(kRows, D, 0, 1) : tc_idesc_bf16(kRows, D, 0, 1);
            const uint64_t q_desc = tc_smem_desc(base + T * L::kQTile, 16, 1024, 2);
            const uint64_t k_desc = tc_smem_desc(base + L::kK, 16, 1024, 2);
            const uint64_t v_desc = tc_smem_desc(base + L::kV, kKVSlab, 1024, 2);
            const uint32_t tS = tmem + T * 256, tO = tS + kOCol;
            // test hook: give up on a barrier that nothing completes
            bool ok = !a.stall_first_wait || wait(stall_bar, 0);
            ok = ok && (FP8 ? wait(q_conv[T], 0) : wait(q_full, 0));
            auto qk = [&](int kb) {
                const int st = kb % kStages;
                ok = ok && wait(kv_full[st], kb / kStages & 1);
                tc_fence_after();
                if (ok) {
                    const uint64_t b0 = k_desc + ((st * L::kStage) >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const int qoff = (kk >> 2) * kQSlab + (kk & 3) * 32, koff = (kk >> 2) * kKVSlab + (kk & 3) * 32;
                        tc_mma_bf16_elect(tS + (kb & 1) * kKeys, q_desc + (qoff >> 4), b0 + (koff >> 4), idesc_qk, kk > 0);
                    }
                }
                tc_commit_elect(smem_addr(&s_full[T][kb & 1]));
            };
            qk(0);
            if (nkb > 1) qk(1);
            for (int kb = 0; kb < nkb; ++kb) {
                const int st = kb % kStages;
                ok = ok && wait(p_full[T][kb & 1], kb >> 1 & 1);
                if (!FP8 && kb == nkb - 1 && partial) ok = ok && wait(v_zeroed, 0);
                tc_fence_after();
                if (ok) {
                    const uint64_t b0 = v_desc + ((st * L::kStage) >> 4);
                    const uint32_t tP = tS + (kb & 1) * kKeys;
#pragma unroll
                    for (int kk = 0; kk < kKeys / 16; ++kk)
                        tc_mma_bf16_ts_elect(tO, tP + kk * 8, b0 + ((kk * 16 * 128) >> 4), idesc_pv, kb > 0 || kk > 0);
                }
                tc_commit_elect(smem_addr(&pv_done[T]));
                tc_commit_elect(smem_addr(&kv_empty[st]));
                if (kb + 2 < nkb) qk(kb + 2);
            }
            if (!ok && lane == 0) fail();
            if (!a.group_start) dependent_release();
            // all is done before the tensor memory is given back
            tc_commit_elect(smem_addr(&drain[T]));
            mbar_wait_suspend(smem_addr(&drain[T]), 0, kDrainNs);
            __syncwarp();
        }
    } else if (warp >= kWiden) {
        if constexpr (FP8) {
            // ---------------- E4M3 to fp16, a row to a thread ----------------
            const int x = warp >= kWiden + 2;  // K or V
            const int r = (warp & 1) * 32 + lane;
            const uint32_t from = base + (x ? L::kRawV : L::kRawK) + r * D, to = base + (x ? L::kV : L::kK) + r * 128;
            bool ok = true;
            for (int kb = 0; kb < nkb; ++kb) {
                const int rs = kb % kRawStages, st = kb % kStages;
                ok = ok && wait(raw_full[x][rs], kb / kRawStages & 1);
                uint4 e[D / 16];
#pragma unroll
                for (int c = 0; c < D / 16; ++c)  // as the copy's swizzle laid it: 128-byte rows, or 64-byte ones
                    e[c] = lds128(from + rs * L::kRaw + ((D == 128 ? c ^ (r & 7) : c ^ (r >> 1 & 3)) << 4));
                const bool valid = kb * kKeys + r < left;
                ok = ok && wait(kv_empty[st], (kb / kStages & 1) ^ 1);
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
                    if (valid) {
                        e4m3x4_to_f16x2x2(e[c].x, lo.x, lo.y);
                        e4m3x4_to_f16x2x2(e[c].y, lo.z, lo.w);
                        e4m3x4_to_f16x2x2(e[c].z, hi.x, hi.y);
                        e4m3x4_to_f16x2x2(e[c].w, hi.z, hi.w);
                    }
                    const int f = 2 * c;  // dims 8 f .. 8 f + 15
                    const uint32_t slab = to + st * L::kStage + (f >> 3) * kKVSlab;
                    st_shared16(slab + (((f & 7) ^ (r & 7)) << 4), lo);
                    st_shared16(slab + ((((f + 1) & 7) ^ (r & 7)) << 4), hi);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_addr(&kv_full[st]));
                    // Not before the stores, which wait for the loads: an arrival does not,
                    // and the next page would land on what is still to be read.
                    mbar_arrive(smem_addr(&raw_empty[x][rs]));
                }
            }
            if (!ok && lane == 0) fail();
        }
    } else {
        // ---------------- softmax: a row to a thread ----------------
        const int T = warp >> 2;
        const int row = (warp & 3) * 32 + lane;
        if (T < ntiles && (warp & 3) < warps_of(T)) {
            const int t = row / a.group, g = row - t * a.group;
            const bool live = t < tokens_of(T);
            const uint32_t tS = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + T * 256, tO = tS + kOCol;
            float scale = a.softmax_log2;
            if constexpr (FP8) scale *= a.k_scales ? a.k_scales[h] : a.kv_scale;
            float m_ref = -INFINITY, l_run = 0.f;
            bool ok = mbar_wait_suspend(smem_addr(&q_full), 0, limit);
            if constexpr (FP8) {  // the row's query to fp16, in place
                for (int sl = 0; sl < L::kSlabs; ++sl)
                    for (int c = 0; c < 8; ++c) {
                        const uint32_t ad = base + T * L::kQTile + sl * kQSlab + row * 128 + ((c ^ (row & 7)) << 4);
                        uint4 x = lds128(ad);
                        x.x = pack2<true>(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u));
                        x.y = pack2<true>(__uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u));
                        x.z = pack2<true>(__uint_as_float(x.z << 16), __uint_as_float(x.z & 0xffff0000u));
                        x.w = pack2<true>(__uint_as_float(x.w << 16), __uint_as_float(x.w & 0xffff0000u));
                        st_shared16(ad, x);
                    }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&q_conv[T]));
            }
            for (int kb = 0; kb < nkb; ++kb) {
                const uint32_t tSb = tS + (kb & 1) * kKeys;  // S(kb), then P(kb)
                ok = ok && mbar_wait_suspend(smem_addr(&s_full[T][kb & 1]), kb >> 1 & 1, limit);
                __syncwarp();
                tc_fence_after();
                float v[64];
                {
                    float lo[32], hi[32];
                    tc_ld32(tSb, lo);
                    tc_ld32(tSb + 32, hi);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        v[i] = lo[i];
                        v[32 + i] = hi[i];
                    }
                }
                if (partial && kb == nkb - 1) {
                    const int n = left - kb * kKeys;
#pragma unroll
                    for (int i = 0; i < 64; ++i) v[i] = i < n ? v[i] : -INFINITY;
                }
                // the largest of the block: four chains of three-input maxima
                float mq[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    mq[q] = fmax3(v[16 * q], v[16 * q + 1], v[16 * q + 2]);
#pragma unroll
                    for (int i = 3; i < 15; i += 2) mq[q] = fmax3(mq[q], v[16 * q + i], v[16 * q + i + 1]);
                    mq[q] = fmaxf(mq[q], v[16 * q + 15]);
                }
                const float top = fmaxf(fmax3(mq[0], mq[1], mq[2]), mq[3]) * scale;  // scale > 0
                bool rescale = false;
                float alpha = 1.f;
                if (top - m_ref > kLazy) {  // the difference: a large score's sum would round
                    alpha = fast_exp2(m_ref - top);
                    m_ref = top;
                    l_run *= alpha;
                    rescale = kb > 0;
                }
                if (__any_sync(0xffffffffu, rescale)) {
                    // O holds PV(kb - 1) before it is scaled; PV(kb) waits for this
                    // block's P, so the barrier is at most a phase away
                    ok = ok && mbar_wait_suspend(smem_addr(&pv_done[T]), (kb - 1) & 1, limit);
                    __syncwarp();
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < D; c += 32) {
                        float o[32];
                        tc_ld32(tO + c, o);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] *= alpha;
                        tc_st32(tO + c, o);
                    }
                    tc_wait_st();
                }
                // no finite score so far: any reference will do for the zeros
                const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
                float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 64; i += 2) {
                    ffma2(v[i], v[i + 1], scale, neg);
                    v[i] = fast_exp2(v[i]);
                    v[i + 1] = fast_exp2(v[i + 1]);
                    fadd2(sa[(i >> 1) & 3], sb[(i >> 1) & 3], v[i], v[i + 1]);
                }
                fadd2(sa[0], sb[0], sa[1], sb[1]);
                fadd2(sa[2], sb[2], sa[3], sb[3]);
                fadd2(sa[0], sb[0], sa[2], sb[2]);
                l_run += sa[0] + sb[0];
                uint32_t pk[32];
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    pk[i] = FP8 ? pack2<true>(v[2 * i] * kRaise, v[2 * i + 1] * kRaise) : pack2<false>(v[2 * i], v[2 * i + 1]);
                tc_st32(tSb, pk);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&p_full[T][kb & 1]));
            }
            ok = ok && mbar_wait_suspend(smem_addr(&drain[T]), 0, limit);
            __syncwarp();
            tc_fence_after();
            if (!ok) fail();
            if (FP8) l_run *= kRaise;
            const int64_t token = static_cast<int64_t>(w.token0) + w.at + T * a.tile_tokens + t;
            const int64_t at = token * a.num_q_heads + h * a.group + g;
            const bool write = live && !failed_s;
            if (a.out) {
                float v_scale = 1.f;
                if constexpr (FP8) v_scale = a.v_scales ? a.v_scales[h] : a.kv_scale;
                const float inv = l_run != 0.f ? v_scale / l_run : 0.f;
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    tc_ld32(tO + c, o);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
                        if (write)
                            *reinterpret_cast<uint4 *>(a.out + at * D + c + i) =
                                make_uint4(pack2<false>(o[i] * inv, o[i + 1] * inv), pack2<false>(o[i + 2] * inv, o[i + 3] * inv),
                                           pack2<false>(o[i + 4] * inv, o[i + 5] * inv), pack2<false>(o[i + 6] * inv, o[i + 7] * inv));
                }
            } else {
                const int64_t slot = w.part * static_cast<int64_t>(a.num_tokens) * a.num_q_heads + at;
                if (write) a.part_ml[slot] = make_float2(m_ref, l_run);
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    tc_ld32(tO + c, o);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        if (write)
                            *reinterpret_cast<float4 *>(a.part_o + slot * D + c + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                }
            }
        }
    }
    // the queries have landed before the CTA ends
    if (tid == 0) mbar_wait_suspend(smem_addr(&q_full), 0, kDrainNs);
    tc_fence_before();
    __syncthreads();
    if (warp == kMma0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

template <int D, bool FP8>
static pa_status launch(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const Args &a, dim3 grid,
                        cudaStream_t stream) {
    using L = Layout<D, FP8>;
    static std::atomic<uint64_t> raised{0};
    pa_status st = sparse::raise_smem_limit(reinterpret_cast<const void *>(rows_kernel<D, FP8>), L::kSmem, raised);
    if (st != PA_OK) return st;
    return cuda_check(launch_dependent(rows_kernel<D, FP8>, grid, L::kThreads, L::kSmem, 0, stream, tq, tk, tv, a),
                      "rows launch");
}

// Least of waves times (a CTA's blocks and its start and end): a block of two full
// tiles takes about 1.1 us, a start and an end 4 us.
int choose_parts(int64_t ctas, int blocks) {
    int best = 1;
    double least = INFINITY;
    for (int parts = 1; parts <= kMaxParts && (parts == 1 || (parts - 1) * kLeastBlocks < blocks); ++parts) {
        const int64_t waves = (ctas * parts + kSms - 1) / kSms;
        const double cost = waves * (4.0 + 1.1 * blocks_per_part(blocks, parts));
        if (cost < least) {
            least = cost;
            best = parts;
        }
    }
    return best;
}

pa_status launch_rows(const void *q, const void *k_cache, const void *v_cache, int head_dim, bool fp8, Args &a,
                      int64_t pairs, int seqs, cudaStream_t stream) {
    a.tile_tokens = kRows / a.group;
    a.wait_limit_ns = wait_limit_ns();
    a.stall_first_wait = stall_first_wait();
    const int64_t pool_rows = static_cast<int64_t>(a.num_blocks) * a.num_kv_heads * a.block_size;
    CUtensorMap tq, tk, tv;
    pa_status st = make_q_map(&tq, q, a.num_tokens, a.num_q_heads, head_dim, a.group, a.tile_tokens);
    if (st == PA_OK) st = make_map(&tk, k_cache, fp8, head_dim, pool_rows, a.block_size);
    if (st == PA_OK) st = make_map(&tv, v_cache, fp8, head_dim, pool_rows, a.block_size);
    if (st != PA_OK) return st;
    if (pairs * a.parts > 0x7fffffff) return fail(PA_ERR_UNSUPPORTED, "too many rows for one launch");
    const dim3 grid(static_cast<unsigned>(pairs * a.parts), a.num_kv_heads, seqs);
    if (head_dim == 128)
        return fp8 ? launch<128, true>(tq, tk, tv, a, grid, stream) : launch<128, false>(tq, tk, tv, a, grid, stream);
    return fp8 ? launch<64, true>(tq, tk, tv, a, grid, stream) : launch<64, false>(tq, tk, tv, a, grid, stream);
}

}  // namespace rows
}  // namespace pa
