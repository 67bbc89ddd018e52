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
// Bound: by the tensor cores and, below their rate, by the chain of a block: scores,
// maximum, powers, product, two blocks of a tile in flight.  16 x 512 rows of 32 / 8 heads
// of 128 dims over 2,048 keys: 212 us, 1,297 TFLOP/s, 0.66 of a library product's rate and
// 0.76 within the loop; a CTA spends some 6.5 us beside it: 1.3 on finding its rows, 0.8 on
// barriers and tensor memory, 1.3 until its queries are there, 1.0 until the first scores are,
// 1.5 on its stores, and 0.5 until the next one starts.  E4M3 pages: 1.1 us a block of two
// tiles where bf16 takes 0.85, for the widening and for 128 registers to a thread.  Small
// tiles are bound by the copies: 32 x 5 rows over up to 4,000 keys, 265 MB, 49.5 us.
//
// Every wait is bounded (2 s unless a test sets another limit).
#include <cudaTypedefs.h>
#include <limits.h>
#include <math.h>

#include <cmath>

#include <atomic>
#include <type_traits>

#include "pa_prefill.cuh"
#include "pa_rows.cuh"
#include "pa_sparse.cuh"

namespace pa {

namespace rows {

constexpr int kKVSlab = kKeys * 128;  // 64 dims of a block's keys or values
constexpr int kTileCols = 256;        // of tensor memory: S at 0 and 64, O at 128
constexpr int kOCol = 128;
constexpr float kLazy = 8.f;
// fp16 probabilities are taken times 2^7: up to 2^15 against the reference's
// 2^8, and whole bits down to 2^-21.
constexpr float kRaise = 128.f;
constexpr uint64_t kDrainNs = 2000000000ull;
constexpr int kMaxSorted = 256;       // sequences that a CTA ranks by length

// Two tiles of 128 rows, one CTA to an SM; or one of up to 64, two CTAs to an SM:
// then the rows are few, the pages' copies are what takes the time, and one CTA's
// begin and end go by under the other's.  (Both kinds' products have 128 rows: of the
// small tile's, the upper ones are whatever lies behind it in shared memory, and
// nobody reads them.)
template <int D, bool FP8, int TILES>
struct Layout {
    static constexpr int kTileRows = tile_rows(TILES);
    static constexpr int kCtas = TILES == 1 ? 2 : 1;
    // warps: the softmax's, 32 rows to each; the copies of K and of V (one warp for
    // both where a tile is alone); the products; the widening of E4M3
    static constexpr int kSoft = TILES * kTileRows / 32;
    static constexpr int kLoadK = kSoft, kMma0 = kSoft + 1;
    static constexpr int kLoadV = TILES == 2 ? kSoft + 2 : kLoadK, kMma1 = TILES == 2 ? kSoft + 3 : -1;
    static constexpr int kWiden = kSoft + 2 * TILES;
    static constexpr int kThreads = 32 * (kWiden + (FP8 ? 4 : 0));
    // Where 512 threads leave 128 registers to each, a row's scores do not stay in them:
    // half of a block's are read again for their powers.  (E4M3, 40 sequences: 148 us, 187
    // with all of them held and more of them spilled; 28 bytes a thread still are with two
    // tiles, 12 with one.)
    static constexpr bool kReread = kThreads * kCtas == 512;
    static constexpr int kSlabs = D / 64;
    static constexpr int kQSlab = kTileRows * 128;  // 64 dims of a tile's queries
    static constexpr int kQTile = kSlabs * kQSlab;
    static constexpr int kStage = kSlabs * kKVSlab;  // a block of K, or of V, as 16-bit rows
    static constexpr int kStages = (TILES == 2 ? (FP8 ? 6 : 10) : FP8 ? 4 : 6) / kSlabs;
    static constexpr int kRaw = kKeys * D;  // a block of E4M3 K, or V
    static constexpr int kRawStages = !FP8 ? 0 : (TILES == 2 ? 8 : 4) / kSlabs;
    static constexpr int kK = TILES * kQTile;
    static constexpr int kV = kK + kStages * kStage;
    static constexpr int kRawK = kV + kStages * kStage;
    static constexpr int kRawV = kRawK + kRawStages * kRaw;
    static constexpr int kBars = kRawV + kRawStages * kRaw;  // the barriers behind it all
    static constexpr int kSmem = kBars + 768;
    static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
};

// Barriers.  kv_full, kv_empty: a stage's K and V are in place, have been read by the
// products of all tiles.  raw_full, raw_empty: E4M3 K (0) and V (1) pages have landed,
// have been read.  q_conv: a tile's queries are fp16.  Of each tile: S(j) is in buffer
// j % 2, P(j) is over it, PV(j) is done, all is done.  stall: never completed.
template <class L, int TILES>
struct Bars {
    static constexpr int kRawStages = L::kRawStages > 0 ? L::kRawStages : 1;
    uint64_t q_full, v_zeroed, stall;
    uint64_t kv_full[L::kStages], kv_empty[L::kStages];
    uint64_t raw_full[2][kRawStages], raw_empty[2][kRawStages];
    uint64_t q_conv[TILES], s_full[TILES][2], p_full[TILES][2], pv_done[TILES], drain[TILES];
    uint32_t tmem_base;
    int failed;
};

// Which rows and which keys a CTA has.
struct Work {
    int token0;  // first token of the rows that the pair's sequence or group has
    int tokens;  // how many it has
    int at;      // the pair's first of them
    int table;   // whose table row leads to the keys
    int keys;    // of the whole run
    int part;
    int head;
};

// Cross attention over runs of unlike lengths: `unit` counts the CTAs that the
// sequences' rows need, those of the longest run first, so that the last to start
// are the shortest, and a sequence without rows has none.  (40 sequences of 0 to 301
// rows and 0 to 2,999 states: a grid of every sequence's most CTAs, in order, left a
// fifth of the SMs' time unused.)  Called by all threads with 4 KB of shared memory;
// every thread comes to the same answer: the sequence, its rows and states, and the
// CTA's place among its CTAs; false for none.  One round of loads for all of it.
template <int TILES>
__device__ __forceinline__ bool longest_unit(const Args &a, int unit, void *room, int &place, Work &w) {
    int *len = static_cast<int *>(room), *order = len + kMaxSorted, *start = order + kMaxSorted;  // kMaxSorted each, and one more
    const int each = TILES * a.tile_tokens, padded = (a.num_seqs + 3) & ~3;
    for (int i = threadIdx.x; i <= a.num_seqs; i += blockDim.x) {
        start[i] = a.query_start[i];
        if (i < a.num_seqs) len[i] = max(a.lens[i], 0);
    }
    for (int i = a.num_seqs + threadIdx.x; i < padded; i += blockDim.x) len[i] = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < a.num_seqs; i += blockDim.x) {
        const int mine = len[i];
        int before = 0;
        for (int j = 0; j < padded; j += 4) {
            const int4 x = *reinterpret_cast<const int4 *>(len + j);
            before += (x.x > mine || (x.x == mine && j < i)) + (x.y > mine || (x.y == mine && j + 1 < i)) +
                      (x.z > mine || (x.z == mine && j + 2 < i)) + (x.w > mine || (x.w == mine && j + 3 < i));
        }
        int count = 0;
        if (query_range(a, start[i], start[i + 1]))
            count = (start[i + 1] - start[i] + each - 1) / each;
        else
            set_device_error(a.err, PA_DEVERR_BAD_CONTEXT);
        order[before] = i | count << 9;  // kMaxSorted is 2^8
    }
    __syncthreads();
    const int lane = threadIdx.x & 31;
    int s = -1;
    for (int i0 = 0; i0 < a.num_seqs && s < 0; i0 += 32) {
        const int x = i0 + lane < a.num_seqs ? order[i0 + lane] : 0;
        int before = x >> 9;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int y = __shfl_up_sync(0xffffffffu, before, d);
            if (lane >= d) before += y;
        }
        const unsigned has = __ballot_sync(0xffffffffu, before > unit);
        const int pick = has ? __ffs(has) - 1 : 31;
        unit -= __shfl_sync(0xffffffffu, before, pick);
        if (has) {
            const int y = __shfl_sync(0xffffffffu, x, pick);
            s = y & 511;
            place = unit + (y >> 9);
        }
    }
    if (s >= 0) {
        w.table = s;
        w.token0 = start[s];
        w.tokens = start[s + 1] - w.token0;
        w.keys = len[s];
    }
    fence_proxy_async_smem();  // copies land in the room next
    __syncthreads();
    return s >= 0;
}

// Called by all threads, which come to the same answer.  False: nothing to do.
template <int TILES>
__device__ __forceinline__ bool find_work(const Args &a, void *room, Work &w) {
    const int lane = threadIdx.x & 31;
    const int cap = a.max_blocks * a.block_size;
    w.head = blockIdx.y;
    if (!a.group_start) {
        int place;
        bool good = true;
        if (a.sorted) {
            const int x = blockIdx.x / a.num_kv_heads, unit = x / a.parts;
            w.head = blockIdx.x - x * a.num_kv_heads;
            w.part = x - unit * a.parts;
            if (!longest_unit<TILES>(a, unit, room, place, w)) return false;
        } else {
            place = blockIdx.x / a.parts;
            w.part = blockIdx.x - place * a.parts;
            w.table = blockIdx.z;
            w.token0 = a.query_start[w.table];
            const int end = a.query_start[w.table + 1];
            good = query_range(a, w.token0, end);
            w.tokens = end - w.token0;
            w.keys = max(a.lens[w.table], 0);
        }
        w.at = TILES * place * a.tile_tokens;
        if (!good || w.keys > cap) {
            if (threadIdx.x == 0) set_device_error(a.err, PA_DEVERR_BAD_CONTEXT);
            w.keys = min(w.keys, cap);
        }
        return good && w.at < w.tokens;
    }
    int pair = blockIdx.x / a.parts;
    w.part = blockIdx.x - pair * a.parts;
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
        const int mine = (hi - lo + TILES * a.tile_tokens - 1) / (TILES * a.tile_tokens);
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
    w.at = TILES * pair * a.tile_tokens;
    w.keys = pages * a.block_size;
    // The table row of the pair's first sequence that has the whole prefix; the
    // others have none of it to themselves, and their rows here are not read.
    const int s0 = first + w.at, s1 = min(end, s0 + TILES * a.tile_tokens);
    w.table = -1;
    for (int s = s0; s < s1 && w.table < 0; s += 32) {
        const int len = s + lane < s1 ? a.lens[s + lane] : 0;
        const unsigned has = __ballot_sync(0xffffffffu, len >= w.keys);
        if (has) w.table = s + __ffs(has) - 1;
    }
    return w.table >= 0;
}

// Groups that are no range of the sequences are reported: a group to a thread, of the CTAs of
// the first KV head.  A CTA looks no further than its own group, so none of them meets all.
__device__ __forceinline__ void check_groups(const Args &a) {
    const int64_t threads = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t g = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; g < a.num_groups; g += threads) {
        const int lo = a.group_start[g], hi = a.group_start[g + 1];
        if (lo < 0 || hi < lo || hi > a.num_seqs) set_device_error(a.err, PA_DEVERR_BAD_CONTEXT);
    }
}

template <int D, bool FP8, int TILES>
__global__ void __launch_bounds__(Layout<D, FP8, TILES>::kThreads, Layout<D, FP8, TILES>::kCtas)
    rows_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const Args a) {
    using L = Layout<D, FP8, TILES>;
    constexpr int kLoadK = L::kLoadK, kLoadV = L::kLoadV, kMma0 = L::kMma0, kMma1 = L::kMma1, kWiden = L::kWiden;
    constexpr uint32_t kTmemCols = TILES * kTileCols;
    constexpr int kStages = L::kStages, kRawStages = FP8 ? L::kRawStages : 1, kQSlab = L::kQSlab;
    // No static shared memory lies in front, so the base is where the swizzle wants it.
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Bars<L, TILES> &bar = *reinterpret_cast<Bars<L, TILES> *>(smem_raw + L::kBars);
    static_assert(sizeof(Bars<L, TILES>) <= L::kSmem - L::kBars, "room for the barriers");

    const uint32_t base = smem_addr(smem_raw);
    const uint64_t limit = a.wait_limit_ns;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    dependent_wait();
    // The kernel that reads a prefix's parts begins with work that needs none of
    // them, and waits for this one's end itself.
    if (a.group_start) dependent_release();
    Work w;
    const bool work = find_work<TILES>(a, smem_raw, w);
    if (a.group_start && blockIdx.y == 0) check_groups(a);  // behind it: the loads are in the cache by now
    if (!work) return;
    const int h = w.head;
    const int all = (w.keys + kKeys - 1) / kKeys, each = blocks_per_part(all, a.parts);
    const int first = w.part * each, nkb = min(each, all - first);  // this part's blocks
    const int ntiles = TILES == 2 && w.at + a.tile_tokens < w.tokens ? 2 : 1;
    auto tokens_of = [&](int T) { return min(a.tile_tokens, w.tokens - w.at - T * a.tile_tokens); };
    auto warps_of = [&](int T) { return (tokens_of(T) * a.group + 31) / 32; };  // with a live row
    if (nkb <= 0) {
        if (a.out && w.keys == 0) {  // nothing to attend to
            const int n = min(w.tokens - w.at, TILES * a.tile_tokens) * a.group * (D / 8);
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
        const int at = TILES == 1 && lane >= pages ? lane - pages : lane;  // K's, then V's
        const int page = (first + kb) * pages + at;
        return at < pages && page * a.block_size < w.keys ? table[page] : kBehind;
    };
    const bool loader = warp == kLoadK || warp == kLoadV;
    const int e_first = loader ? page_entry(0) : kBehind;

    if (warp == 0) {  // a barrier to a lane: one lane alone takes as long as the first table entry
        auto init = [&](uint64_t *bars, int n, int count) {
            if (lane < n) mbar_init(smem_addr(bars + lane), count);
        };
        init(&bar.q_full, 3, 1);  // and v_zeroed, stall
        init(bar.kv_full, kStages, FP8 ? 4 : TILES);  // the widening warps, or the loaders
        init(bar.kv_empty, kStages, ntiles);          // those that read the block
        if constexpr (FP8) {
            init(bar.raw_full[0], 2 * kRawStages, 1);
            init(bar.raw_empty[0], 2 * kRawStages, 2);
        }
        init(bar.s_full[0], 2 * TILES, 1);
        for (int T = 0; T < TILES; ++T) init(bar.p_full[T], 2, T < ntiles ? warps_of(T) : 1);
        init(bar.pv_done, TILES, 1);
        init(bar.drain, TILES, 1);
        for (int T = 0; T < TILES; ++T) init(bar.q_conv + T, 1, T < ntiles ? warps_of(T) : 1);
        fence_barrier_init();
        __syncwarp();
    }
    if (tid == 0) {
        bar.failed = 0;
        const int q_box = D * 2 * a.group * a.tile_tokens;
        mbar_arrive_expect_tx(smem_addr(&bar.q_full), ntiles * q_box);
        for (int T = 0; T < ntiles; ++T)
            for (int sl = 0; sl < L::kSlabs; ++sl)
                tma_load_3d(base + T * L::kQTile + sl * kQSlab, &tmQ, sl * 64, h * a.group,
                            w.token0 + w.at + T * a.tile_tokens, smem_addr(&bar.q_full));
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (warp == kMma0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&bar.tmem_base)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem_base;
    auto fail = [&]() {
        set_device_error(a.err, PA_DEVERR_TIMEOUT);
        atomicExch(&bar.failed, 1);
    };
    // a whole warp waits
    auto wait = [&](uint64_t &b, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait_suspend(smem_addr(&b), parity, limit)) != 0;
    };

    if (loader) {
        // ---------------- copies of pages ----------------
        // K (0) or V (1), or the first and the second half of the lanes that have a page
        constexpr bool kBoth = TILES == 1;
        const int x = kBoth ? (lane >= pages) : warp != kLoadK, page = kBoth && lane >= pages ? lane - pages : lane;
        const int rows_total = a.num_blocks * a.num_kv_heads * a.block_size;
        const CUtensorMap *map = x == 0 ? &tmK : &tmV;
        const uint64_t policy = l2_evict_first_policy();
        constexpr int kRing = FP8 ? kRawStages : kStages;
        constexpr int kBytes = FP8 ? L::kRaw : L::kStage;
        const uint32_t ring = base + (FP8 ? (x == 0 ? L::kRawK : L::kRawV) : (x == 0 ? L::kK : L::kV));
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
            const uint32_t parity = (kb / kRing & 1) ^ 1;
            bool freed;
            uint64_t *full;  // of this lane's page
            if constexpr (FP8) {
                freed = wait(bar.raw_empty[kBoth ? 0 : x][st], parity);
                if (kBoth) freed = wait(bar.raw_empty[1][st], parity) && freed;
                full = &bar.raw_full[x][st];
            } else {
                freed = wait(bar.kv_empty[st], parity);
                full = &bar.kv_full[st];
            }
            if (lane == 0) {
                if (!freed) fail();
                mbar_arrive_expect_tx(smem_addr(full), kBoth && !FP8 ? 2 * kBytes : kBytes);
                if (kBoth && FP8) mbar_arrive_expect_tx(smem_addr(&bar.raw_full[1][st]), kBytes);
            }
            __syncwarp();
            if (lane < (kBoth ? 2 * pages : pages)) {
                if constexpr (FP8) {
                    tma_load_2d(ring + st * kBytes + page * a.block_size * D, map, 0, y, smem_addr(full), policy);
                } else {
                    for (int sl = 0; sl < L::kSlabs; ++sl)
                        tma_load_2d(ring + st * kBytes + sl * kKVSlab + page * a.block_size * 128, map, sl * 64, y,
                                    smem_addr(full), policy);
                }
            }
        }
        if (!FP8 && warp == kLoadV && partial) {
            const int kb = nkb - 1, st = kb % kStages;
            if (!wait(bar.kv_full[st], kb / kStages & 1) && lane == 0) fail();
            for (int r = left - kb * kKeys + lane; r < kKeys; r += 32)
                for (int sl = 0; sl < L::kSlabs; ++sl)
                    for (int c = 0; c < 8; ++c) st_shared_zero16(base + L::kV + st * L::kStage + sl * kKVSlab + r * 128 + c * 16);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&bar.v_zeroed));
        }
        // whatever gave up, the CTA ends after its copies: those of the last blocks may be in flight
        if (lane == 0)
            for (int kb = max(0, nkb - kRing); kb < nkb; ++kb) {
                if constexpr (FP8) {
                    mbar_wait_suspend(smem_addr(&bar.raw_full[kBoth ? 0 : x][kb % kRing]), kb / kRing & 1, kDrainNs);
                    if (kBoth) mbar_wait_suspend(smem_addr(&bar.raw_full[1][kb % kRing]), kb / kRing & 1, kDrainNs);
                } else {
                    mbar_wait_suspend(smem_addr(&bar.kv_full[kb % kRing]), kb / kRing & 1, kDrainNs);
                }
            }
    } else if (warp == kMma0 || warp == kMma1) {
        // ---------------- products ----------------
        const int T = warp == kMma0 ? 0 : 1;
        if (T < ntiles) {
            constexpr uint32_t idesc_qk = FP8 ? tc_idesc_f16(kRows, kKeys, 0, 0) : tc_idesc_bf16(kRows, kKeys, 0, 0);
            constexpr uint32_t idesc_pv = FP8 ? tc_idesc_f16(kRows, D, 0, 1) : tc_idesc_bf16(kRows, D, 0, 1);
            const uint64_t q_desc = tc_smem_desc(base + T * L::kQTile, 16, 1024, 2);
            const uint64_t k_desc = tc_smem_desc(base + L::kK, 16, 1024, 2);
            const uint64_t v_desc = tc_smem_desc(base + L::kV, kKVSlab, 1024, 2);
            const uint32_t tS = tmem + T * kTileCols, tO = tS + kOCol;
            // test hook: give up on a barrier that nothing completes
            bool ok = !a.stall_first_wait || wait(bar.stall, 0);
            ok = ok && (FP8 ? wait(bar.q_conv[T], 0) : wait(bar.q_full, 0));
            auto qk = [&](int kb) {
                const int st = kb % kStages;
                ok = ok && wait(bar.kv_full[st], kb / kStages & 1);
                tc_fence_after();
                if (ok) {
                    const uint64_t b0 = k_desc + ((st * L::kStage) >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const int qoff = (kk >> 2) * kQSlab + (kk & 3) * 32, koff = (kk >> 2) * kKVSlab + (kk & 3) * 32;
                        tc_mma_bf16_elect(tS + (kb & 1) * kKeys, q_desc + (qoff >> 4), b0 + (koff >> 4), idesc_qk, kk > 0);
                    }
                }
                tc_commit_elect(smem_addr(&bar.s_full[T][kb & 1]));
            };
            qk(0);
            if (nkb > 1) qk(1);
            for (int kb = 0; kb < nkb; ++kb) {
                const int st = kb % kStages;
                ok = ok && wait(bar.p_full[T][kb & 1], kb >> 1 & 1);
                if (!FP8 && kb == nkb - 1 && partial) ok = ok && wait(bar.v_zeroed, 0);
                tc_fence_after();
                if (ok) {
                    const uint64_t b0 = v_desc + ((st * L::kStage) >> 4);
                    const uint32_t tP = tS + (kb & 1) * kKeys;
#pragma unroll
                    for (int kk = 0; kk < kKeys / 16; ++kk)
                        tc_mma_bf16_ts_elect(tO, tP + kk * 8, b0 + ((kk * 16 * 128) >> 4), idesc_pv, kb > 0 || kk > 0);
                }
                tc_commit_elect(smem_addr(&bar.pv_done[T]));
                tc_commit_elect(smem_addr(&bar.kv_empty[st]));
                if (kb + 2 < nkb) qk(kb + 2);
            }
            if (!ok && lane == 0) fail();
            if (!a.group_start) dependent_release();
            // all is done before the tensor memory is given back
            tc_commit_elect(smem_addr(&bar.drain[T]));
            mbar_wait_suspend(smem_addr(&bar.drain[T]), 0, kDrainNs);
            __syncwarp();
        }
    } else if (warp >= kWiden) {
        if constexpr (FP8) {
            // ---------------- E4M3 to fp16, a row to a thread ----------------
            const int x = warp >= kWiden + 2;  // K or V
            const int r = (warp - kWiden & 1) * 32 + lane;
            const uint32_t from = base + (x ? L::kRawV : L::kRawK) + r * D, to = base + (x ? L::kV : L::kK) + r * 128;
            bool ok = true;
            for (int kb = 0; kb < nkb; ++kb) {
                const int rs = kb % kRawStages, st = kb % kStages;
                ok = ok && wait(bar.raw_full[x][rs], kb / kRawStages & 1);
                uint4 e[D / 16];
#pragma unroll
                for (int c = 0; c < D / 16; ++c)  // as the copy's swizzle laid it: 128-byte rows, or 64-byte ones
                    e[c] = lds128(from + rs * L::kRaw + ((D == 128 ? c ^ (r & 7) : c ^ (r >> 1 & 3)) << 4));
                const bool valid = kb * kKeys + r < left;
                ok = ok && wait(bar.kv_empty[st], (kb / kStages & 1) ^ 1);
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
                    mbar_arrive(smem_addr(&bar.kv_full[st]));
                    // Not before the stores, which wait for the loads: an arrival does not,
                    // and the next page would land on what is still to be read.
                    mbar_arrive(smem_addr(&bar.raw_empty[x][rs]));
                }
            }
            if (!ok && lane == 0) fail();
        }
    } else {
        // ---------------- softmax: a row to a thread ----------------
        const int T = TILES == 1 ? 0 : warp >> 2, quarter = TILES == 1 ? warp : warp & 3;
        const int row = quarter * 32 + lane;
        if (T < ntiles && quarter < warps_of(T)) {
            const int t = row / a.group, g = row - t * a.group;
            const uint32_t tS = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + T * kTileCols, tO = tS + kOCol;
            float scale = a.softmax_log2;
            if constexpr (FP8) scale *= a.k_scales ? a.k_scales[h] : a.kv_scale;
            float m_ref = -INFINITY, l_run = 0.f;
            bool ok = mbar_wait_suspend(smem_addr(&bar.q_full), 0, limit);
            // The row's query to fp16, in place: K is fp16, which holds all E4M3 values, and a
            // product's two sides have one type.  Exact between 2^-17 and 65,504.
            if constexpr (FP8) {
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
                if (lane == 0) mbar_arrive(smem_addr(&bar.q_conv[T]));
            }
            for (int kb = 0; kb < nkb; ++kb) {
                const uint32_t tSb = tS + (kb & 1) * kKeys;  // S(kb), then P(kb)
                ok = ok && mbar_wait_suspend(smem_addr(&bar.s_full[T][kb & 1]), kb >> 1 & 1, limit);
                __syncwarp();
                tc_fence_after();
                // scores 32 half .. of the row, masked behind the run's end
                auto scores = [&](int half, float (&x)[32]) {
                    tc_ld32(tSb + 32 * half, x);
                    tc_wait_ld();
                    if (partial && kb == nkb - 1) {
                        const int n = left - kb * kKeys - 32 * half;
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = i < n ? x[i] : -INFINITY;
                    }
                };
                // their largest: two chains of three-input maxima
                auto largest = [](const float (&x)[32]) {
                    float m[2];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        m[q] = fmax3(x[16 * q], x[16 * q + 1], x[16 * q + 2]);
#pragma unroll
                        for (int i = 3; i < 15; i += 2) m[q] = fmax3(m[q], x[16 * q + i], x[16 * q + i + 1]);
                    }
                    return fmax3(m[0], m[1], fmaxf(x[15], x[31]));
                };
                float lo[32], hi[32];
                if constexpr (L::kReread) {
                    scores(0, lo);
                } else {  // both loads in flight
                    tc_ld32(tSb, lo);
                    tc_ld32(tSb + 32, hi);
                    tc_wait_ld();
                    if (partial && kb == nkb - 1) {
                        const int n = left - kb * kKeys;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            lo[i] = i < n ? lo[i] : -INFINITY;
                            hi[i] = 32 + i < n ? hi[i] : -INFINITY;
                        }
                    }
                }
                float top = largest(lo);
                if constexpr (L::kReread) scores(1, hi);
                top = fmaxf(top, largest(hi)) * scale;  // scale > 0
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
                    ok = ok && mbar_wait_suspend(smem_addr(&bar.pv_done[T]), (kb - 1) & 1, limit);
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
                // The sum takes the powers as they are, the product as 16 bits, of V's type as
                // it has to: one bf16 number, off by up to 2^-8 of it (an output's error is 0.0023
                // of its norm, 0.0017 by the output's own rounding alone), or one fp16 number, up
                // to 2^-11 (0.0017 as well).  The list kernel keeps what the bf16 number leaves as
                // a second one and is bound by memory; here that is half as many products again.
                uint32_t pk[32];
                auto powers = [&](int half, float (&x)[32]) {
                    float sa[2] = {0.f, 0.f}, sb[2] = {0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        ffma2(x[i], x[i + 1], scale, neg);
                        x[i] = fast_exp2(x[i]);
                        x[i + 1] = fast_exp2(x[i + 1]);
                        fadd2(sa[(i >> 1) & 1], sb[(i >> 1) & 1], x[i], x[i + 1]);
                        pk[16 * half + i / 2] = FP8 ? pack2<true>(x[i] * kRaise, x[i + 1] * kRaise) : pack2<false>(x[i], x[i + 1]);
                    }
                    fadd2(sa[0], sb[0], sa[1], sb[1]);
                    l_run += sa[0] + sb[0];
                };
                powers(1, hi);
                if constexpr (L::kReread) scores(0, lo);
                powers(0, lo);
                tc_st32(tSb, pk);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&bar.p_full[T][kb & 1]));
            }
            ok = ok && mbar_wait_suspend(smem_addr(&bar.drain[T]), 0, limit);
            __syncwarp();
            tc_fence_after();
            if (!ok) fail();
            if (FP8) l_run *= kRaise;
            const int64_t first_row = (static_cast<int64_t>(w.token0) + w.at + T * a.tile_tokens) * a.num_q_heads + h * a.group;
            const int mine = t * a.num_q_heads + g;  // from there to this lane's row
            // Rows leave through shared memory, each warp's 32 through the space of their
            // queries: whole rows to a store instruction (a row to a lane would be
            // 32 pieces of 16 bytes in as many lines).  The tile's products are done with it.
            const uint32_t stage = base + T * L::kQTile + quarter * (L::kQTile * 32 / L::kTileRows);
            constexpr int kRowBytes = 2 * D, kPieces = kRowBytes / 16, kAtOnce = 32 / kPieces;
            const int rows_here = bar.failed ? 0 : min(32, tokens_of(T) * a.group - quarter * 32);
            auto put = [&](int c, const uint4 &x) {  // 16-byte piece c of this lane's row
                st_shared16(stage + lane * kRowBytes + (((c & ~7) | ((c ^ lane) & 7)) << 4), x);
            };
            auto flush = [&](char *to, int64_t row_stride) {  // the warp's rows, each to its place from `to` on
                __syncwarp();
#pragma unroll 4
                for (int r0 = 0; r0 < rows_here; r0 += kAtOnce) {
                    const int r = r0 + lane / kPieces, c = lane % kPieces;
                    const int64_t row = __shfl_sync(0xffffffffu, mine, r);
                    const uint4 x = lds128(stage + r * kRowBytes + (((c & ~7) | ((c ^ r) & 7)) << 4));
                    if (r < rows_here) *reinterpret_cast<uint4 *>(to + row * row_stride + c * 16) = x;
                }
                __syncwarp();
            };
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
                        put((c + i) / 8, make_uint4(pack2<false>(o[i] * inv, o[i + 1] * inv), pack2<false>(o[i + 2] * inv, o[i + 3] * inv),
                                                    pack2<false>(o[i + 4] * inv, o[i + 5] * inv), pack2<false>(o[i + 6] * inv, o[i + 7] * inv)));
                }
                flush(reinterpret_cast<char *>(a.out + first_row * D), kRowBytes);
            } else {
                const int64_t slot = w.part * static_cast<int64_t>(a.num_tokens) * a.num_q_heads + first_row;
                if (lane < rows_here) a.part_ml[slot + mine] = make_float2(m_ref, l_run);
#pragma unroll
                for (int half = 0; half < 2; ++half) {  // 2 D bytes are half a row's
#pragma unroll
                    for (int c = 0; c < D / 2; c += 32) {
                        float o[32];
                        tc_ld32(tO + half * (D / 2) + c, o);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            put((c + i) / 4, make_uint4(__float_as_uint(o[i]), __float_as_uint(o[i + 1]), __float_as_uint(o[i + 2]),
                                                        __float_as_uint(o[i + 3])));
                    }
                    flush(reinterpret_cast<char *>(a.part_o + slot * D + half * (D / 2)), 4 * D);
                }
            }
        }
    }
    // the queries have landed before the CTA ends
    if (tid == 0) mbar_wait_suspend(smem_addr(&bar.q_full), 0, kDrainNs);
    tc_fence_before();
    __syncthreads();
    if (warp == kMma0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

template <int D, bool FP8, int TILES>
static pa_status launch(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const Args &a, dim3 grid,
                        cudaStream_t stream) {
    using L = Layout<D, FP8, TILES>;
    static std::atomic<uint64_t> raised{0};
    pa_status st = sparse::raise_smem_limit(reinterpret_cast<const void *>(rows_kernel<D, FP8, TILES>), L::kSmem, raised);
    if (st != PA_OK) return st;
    return cuda_check(launch_dependent(rows_kernel<D, FP8, TILES>, grid, L::kThreads, L::kSmem, 0, stream, tq, tk, tv, a),
                      "rows launch");
}

// Microseconds of a CTA over `blocks` blocks, its start and end among them.
double cta_time(int blocks, int tiles, int head_dim) {
    return tiles == 1 ? 3.0 + (head_dim == 64 ? 0.85 : 1.4) * blocks : 4.0 + (head_dim == 64 ? 0.6 : 0.9) * blocks;
}

// Writing and reading `parts` parts.
double join_time(int parts, int head_dim, int64_t num_rows) {
    return parts * (static_cast<double>(num_rows) * head_dim * 8) / 5e6;
}

// Least of an estimated time.  Runs of one length (`even`) end in whole waves.  Of
// others 0.6 or 0.65 of the longest is taken for the average, and the work is shared out:
// where one part needs no joining (cross attention) the longest run first, and what
// remains of it at the end has its SM to itself; else in their order, and the last CTA
// is half done when the others end.  (32 sequences of up to 4,000 states, 5 rows of 32 / 8
// heads: 61.3 us with one part, 50.2 with two, 57.2 with three; 100 sequences 131 with
// one, 165 with two; 8 sequences 53 with one, 20.8 with five, 24.1 with eight; 26 of up to 452
// states, 6 rows, 11.5 with one, 15.0 with two.)
int choose_parts(int64_t ctas, int blocks, int tiles, int head_dim, int64_t num_rows, bool even, bool direct) {
    const int64_t places = tiles == 1 ? 2 * kSms : kSms;
    int best = 1;
    double least = INFINITY;
    for (int parts = 1; parts <= kMaxParts && (parts == 1 || (parts - 1) * kLeastBlocks < blocks); ++parts) {
        const double one = cta_time(blocks_per_part(blocks, parts), tiles, head_dim), n = static_cast<double>(ctas) * parts;
        const double start = cta_time(0, tiles, head_dim), work = ctas * (cta_time(blocks, tiles, head_dim) - start);
        double cost;
        if (even)
            cost = std::ceil(n / places) * one;
        else if (direct)
            cost = std::max(start + (one - start) * (tiles == 1 ? 0.65 : 1.0), (n * start + work * 0.65) / places);
        else
            cost = std::max(one, (n * start + work * 0.6) / places + one / 2);
        if (parts > 1 || !direct) cost += join_time(parts, head_dim, num_rows) + (direct ? 3.0 : 0.0);  // a kernel more
        if (cost < least) {
            least = cost;
            best = parts;
        }
    }
    return best;
}

pa_status launch_rows(const void *q, const void *k_cache, const void *v_cache, int head_dim, bool fp8, Args &a,
                      int tiles, int64_t ctas, int seqs, cudaStream_t stream) {
    a.tile_tokens = tile_rows(tiles) / a.group;
    a.wait_limit_ns = wait_limit_ns();
    a.stall_first_wait = stall_first_wait();
    const int64_t pool_rows = static_cast<int64_t>(a.num_blocks) * a.num_kv_heads * a.block_size;
    CUtensorMap tq, tk, tv;
    pa_status st = make_q_map(&tq, q, a.num_tokens, a.num_q_heads, head_dim, a.group, a.tile_tokens);
    if (st == PA_OK) st = make_map(&tk, k_cache, fp8, head_dim, pool_rows, a.block_size);
    if (st == PA_OK) st = make_map(&tv, v_cache, fp8, head_dim, pool_rows, a.block_size);
    if (st != PA_OK) return st;
    dim3 grid(1, a.num_kv_heads, seqs);
    int64_t x = ctas * a.parts;
    // A few waves or more of CTAs, of sequences that a CTA can sort: by length.
    a.sorted = !a.group_start && seqs > 1 && seqs <= kMaxSorted && x * a.num_kv_heads * seqs > kSms &&
               ctas < 1 << 22;  // a sequence's place and CTAs share a word
    if (a.sorted) {
        const int64_t each = static_cast<int64_t>(tiles) * a.tile_tokens;
        x = std::min(ctas * seqs, a.num_tokens / each + seqs) * a.parts * a.num_kv_heads;
        grid.y = grid.z = 1;
    }
    if (x > 0x7fffffff) return fail(PA_ERR_UNSUPPORTED, "too many rows for one launch");
    grid.x = static_cast<unsigned>(x);
    auto shape = [&](auto d, auto t) {
        return fp8 ? launch<d.value, true, t.value>(tq, tk, tv, a, grid, stream)
                   : launch<d.value, false, t.value>(tq, tk, tv, a, grid, stream);
    };
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I64 = std::integral_constant<int, 64>;
    using I128 = std::integral_constant<int, 128>;
    if (head_dim == 128) return tiles == 1 ? shape(I128{}, I1{}) : shape(I128{}, I2{});
    return tiles == 1 ? shape(I64{}, I1{}) : shape(I64{}, I2{});
}

}  // namespace rows
}  // namespace pa
