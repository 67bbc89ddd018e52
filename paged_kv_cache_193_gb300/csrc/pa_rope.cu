// Rotate-and-append: the position rotation of a batch of new tokens' q and k
// rows, and the write of their k and v rows into the paged cache, in one
// kernel ("Optimizing Llama 3.1 405B Inference with vLLM PagedAttention",
// section "PagedAttention Mechanics": a token's K and V are appended on
// arrival; the pages leave the rotation to the model).  For models that
// normalise every head's q and k first, that is done on the way (NORM).
//
// Mathematics: pair i of a row (x_a, x_b) is turned by the angle
// theta = position * inv_freq[i]:
//   x'_a = m (x_a cos theta - x_b sin theta)
//   x'_b = m (x_a sin theta + x_b cos theta)
// The angle is reduced in whole numbers: inv_freq / 2 pi, taken modulo one
// turn, is held as a 64-bit fraction F of a turn, and position * F modulo 2^64
// is the angle as a fraction of a turn with no rounding in the product.  F is off
// by at most 2^-64 turns plus 2^-61 inv_freq, so the angle by |position| times
// that: below 2^-29 turns at any position for frequencies up to 1.  Its upper 32
// bits go to sine and cosine as an fp32 number of half turns, within 2^-24.
//
// NORM: a row of q or k becomes x * rsqrt(mean x^2 + eps) * (offset + w) before it
// is turned, all in fp32 and rounded once with the rotation.  A row is in the
// registers of head_dim / 16 neighbouring lanes, so its sum of squares takes two or
// three shuffles and no pass of its own over memory.
//
// Bound: memory.  Every q, k, v element is read once and written once: 8192
// tokens of 32 query and 8 KV heads, 201 MB, take 32.5 us, with NORM 34.3, where a
// library copy of as much takes 32.5; few tokens are bound by the launch (one: 2.0
// and 2.4 us) and by the chain position, sine and cosine, row, so a thread's first rows
// are on their way while the angles are made.
#include <algorithm>
#include <cstring>
#include <tuple>
#include <utility>

#include "pa_launch.cuh"

namespace pa {
namespace rope {

// How x / scale is found where only its E4M3 code matters: x times RN(1 /
// scale) is within two units in the last place of RN(x / scale), so both have
// the same code unless a border between two codes is that near, and then the
// division decides (Ziv's rounding test, "Fast evaluation of elementary
// mathematical functions with correctly rounded last bit", 1991).  The borders,
// and the codes, have at most five significant bits, so near them the lower 19
// of a float's are almost all 0 or almost all 1.  Below 2^-126 and above 448 the
// code is 0 or the largest, whatever the last place.  (8192 tokens, 32 + 8 heads,
// when all rows still came by registers: 36.5 us with it, 39.5 with a division for
// every element; 256 tokens of 64 + 8 heads 3.7 and 4.0.)
struct Divisor {
    float scale, inverse;
    // Of the 2^19 endings of a product, how many are in doubt, times 2^13: none when
    // the product is exact, all when 1 / scale may be out of range.
    uint32_t near;
    __host__ __device__ __forceinline__ static Divisor of(float x) {
        const bool all = !(x >= 7.888609052210118e-31f && x <= 1.2676506002282294e30f);  // 2^-100, 2^100
        uint32_t bits;
        memcpy(&bits, &x, 4);
        return {x, 1.f / x, all ? 0xffffffffu : bits & 0x7fffff ? 9u << 13 : 0u};
    }
};

struct Args {
    const __nv_bfloat16 *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements between tokens
    const int32_t *positions;              // [axes][num_tokens]
    const double *inv_freq;                // [rotary_dim / 2]
    const int32_t *pair_axis;              // [rotary_dim / 2] or null (axis 0)
    const int32_t *slots;
    __nv_bfloat16 *q_out;
    uint8_t *k_cache, *v_cache;
    int64_t num_slots;
    int num_tokens, num_axes, num_q_heads, num_kv_heads, block_size;
    int pairs;       // rotary_dim / 2
    int tile;        // tokens per CTA
    int rows_per_y;  // rows (of one token's q, k and v heads) per CTA
    float magnitude;
    Divisor kv_scale;
    const float *k_scales, *v_scales;
    unsigned int *err;
    // NORM: bf16 weights of head 0, or null (1), elements between heads' weights
    const __nv_bfloat16 *q_weight, *k_weight;
    int64_t q_weight_stride, k_weight_stride;
    float weight_offset, eps;
};

constexpr int kThreads = 256;
constexpr int kMaxTile = 8;

__device__ __forceinline__ void unpack8(const uint4 &w, float2 (&x)[4]) {
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __bfloat1622float2(h[i]);
}

__device__ __forceinline__ uint4 pack8(const float2 (&x)[4]) {
    return make_uint4(pack2<false>(x[0].x, x[0].y), pack2<false>(x[1].x, x[1].y), pack2<false>(x[2].x, x[2].y),
                      pack2<false>(x[3].x, x[3].y));
}

// Two fp32 products, sums or fused multiply-adds in one instruction, each rounded
// as by itself.
__device__ __forceinline__ float2 mul2(float2 x, float2 y) { return __fmul2_rn(x, y); }
__device__ __forceinline__ float2 add2(float2 x, float2 y) { return __fadd2_rn(x, y); }
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) { return __ffma2_rn(x, y, z); }

// Where entry p of a table in shared memory lies that is read in groups of eight: the
// first halves of all groups, then the second, so that lanes that read a group each
// find their 16 bytes side by side.
template <int N>
__device__ __forceinline__ constexpr int spread(int p) {
    return (p & 4) * (N / 8) + (p >> 3) * 4 + (p & 3);
}
template <int N>
__device__ __forceinline__ void take8(const float *table, int group, float2 (&x)[4]) {
    const float4 lo = *reinterpret_cast<const float4 *>(table + 4 * group), hi = *reinterpret_cast<const float4 *>(table + N / 2 + 4 * group);
    x[0] = make_float2(lo.x, lo.y);
    x[1] = make_float2(lo.z, lo.w);
    x[2] = make_float2(hi.x, hi.y);
    x[3] = make_float2(hi.z, hi.w);
}

// f / 2 pi modulo one turn, as a 64-bit fraction of a turn, from the bits of f
// (the fp64 unit is some sixty times slower than the integer one here): the
// significand times 2 / pi, of which the upper 64 bits are kept, shifted by the
// exponent.  Off by less than 2^-64 turns plus 2^-61 of f; 0 for what is not
// finite and from 2^65 on.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
    const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(f));
    const int exponent = static_cast<int>(bits >> 52 & 0x7ff) - 1023;  // f = 1.m * 2^exponent
    const uint64_t significand = (bits | 1ull << 52) << 11;            // 1.m * 2^63
    // 2 / pi * 2^64, rounded; the product is 1.m * 2 / pi * 2^63
    const uint64_t part = __umul64hi(significand, 0xa2f9836e4e44152aull);
    const int shift = exponent - 1;  // to f / 2 pi * 2^64
    const uint64_t turn = shift <= -64 || shift >= 64 ? 0 : shift >= 0 ? part << shift : part >> -shift;
    return bits >> 63 ? 0ull - turn : turn;
}

// Eight fp32 values as E4M3 codes of x / scale: one rounding from fp32 (the
// rotated row is not rounded to bf16 on the way).
__device__ __forceinline__ uint2 codes8(const float2 (&x)[4], const Divisor &by) {
    uint32_t w[2] = {0, 0};
    uint32_t least = 0xffffffffu;  // of the endings, plus 4, in the upper 19 bits
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 y = make_float2(__fmul_rn(x[i / 2].x, by.inverse), __fmul_rn(x[i / 2].y, by.inverse));
        least = min(least, min(__float_as_uint(y.x) * 8192u + 32768u, __float_as_uint(y.y) * 8192u + 32768u));
        w[i / 4] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3)) << 8 * (i % 4);
    }
    if (least < by.near) {
        w[0] = w[1] = 0;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float2 y = make_float2(__fdiv_rn(x[i / 2].x, by.scale), __fdiv_rn(x[i / 2].y, by.scale));
            w[i / 4] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3)) << 8 * (i % 4);
        }
    }
    return make_uint2(w[0], w[1]);
}

// A thread works on 16 elements of one head's row at a time, two vectors of eight:
// with pairs (i, i + R/2) elements 8j .. 8j+7 and their partners, otherwise those
// from 8j and from D/2 + 8j on, so that the lanes' 16 bytes lie side by side.  Its j is
// the same for every row it takes.  Its first row comes by registers, the next by
// shared memory, where two more are on their way while it works on one: 8192 tokens, 32 +
// 8 heads, 32.5 us, in E4M3 31.3, with NORM 34.3; with the next row asked for when one is
// done 34.5, 36.5 and 42.2; with one more on its way 33.7 and (NORM) 37.0, with three
// 32.3 and 37.4, each at five CTAs to an SM.
// NORM: none, with weights (or none) that all heads share, which are kept in shared
// memory, or with each head's own.  CTAS: of the kernel to an SM, which caps its
// registers.
enum { kNone, kShared, kHeads };
template <int D, bool FP8, bool ADJACENT, int NORM, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS) append_kernel(const Args a) {
    constexpr int VPR = D / 16;  // threads to a row
    __shared__ __align__(16) float cs[kMaxTile][D / 2], sn[kMaxTile][D / 2];
    __shared__ int64_t row_s[kMaxTile];  // the slot's row of head 0, or -1
    // weights that all heads have, with the offset: q's, then k's
    __shared__ __align__(16) float weight_s[NORM == kShared ? 2 : 1][NORM == kShared ? D : 1];
    dependent_wait();
    const int t0 = blockIdx.x * a.tile;
    const int live = min(a.tile, a.num_tokens - t0);
    const int j = threadIdx.x % VPR;
    const int rows = a.num_q_heads + 2 * a.num_kv_heads;
    const int row0 = blockIdx.y * a.rows_per_y;
    const int nrows = min(a.rows_per_y, rows - row0);
    // which of the thread's two vectors are turned, and their first elements
    const bool turn = ADJACENT ? 8 * j < 2 * a.pairs : 8 * j < a.pairs, turn_b = ADJACENT ? D / 2 + 8 * j < 2 * a.pairs : turn;
    const int ea = ADJACENT || turn ? 8 * j : a.pairs + 8 * j;
    const int eb = ADJACENT || !turn ? D / 2 + 8 * j : a.pairs + 8 * j;
    // Pieces behind the first, kPieces - 1 of them on their way: each lands in the thread's
    // own place, so no barrier is needed, and the one that is written to was used the turn before.
    // With weights of each head's own these come beside their row.
    constexpr int kPieces = NORM == kHeads ? 2 : 3;
    __shared__ __align__(16) uint4 piece[kPieces][NORM == kHeads ? 4 : 2][kThreads];
    uint4 ga, gb;  // the present one's weights
    uint4 wa, wb;  // the present one
    const int first = threadIdx.x / VPR;
    int tt = first / nrows, at = first - tt * nrows;  // its token and row
    int next_tt = tt, next_at = at;                   // of the next to be fetched
    int h;
    bool is_q, is_v;
    auto what = [&](int at) {
        const int row = row0 + at;
        is_q = row < a.num_q_heads;
        is_v = row >= a.num_q_heads + a.num_kv_heads;
        h = row - (is_q ? 0 : is_v ? a.num_q_heads + a.num_kv_heads : a.num_q_heads);
    };
    auto advance = [&](int &tt, int &at) {
        for (at += kThreads / VPR; at >= nrows; at -= nrows) ++tt;
    };
    auto source = [&](int tt) {
        const int64_t t = t0 + tt;
        return (is_q ? a.q + t * a.q_stride : is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride) + static_cast<int64_t>(h) * D;
    };
    auto weights = [&]() -> const __nv_bfloat16 * {  // the head's own, if any
        const __nv_bfloat16 *weight = NORM != kHeads || is_v ? nullptr : is_q ? a.q_weight : a.k_weight;
        return weight ? weight + h * (is_q ? a.q_weight_stride : a.k_weight_stride) : nullptr;
    };
    auto fetch = [&](int place) {
        if (next_tt < live) {
            what(next_at);
            const __nv_bfloat16 *src = source(next_tt);
            cp_async16(smem_addr(&piece[place][0][threadIdx.x]), src + (is_v ? 8 * j : ea));
            cp_async16(smem_addr(&piece[place][1][threadIdx.x]), src + (is_v ? D / 2 + 8 * j : eb));
            if (const __nv_bfloat16 *weight = weights()) {
                cp_async16_l1(smem_addr(&piece[place][2][threadIdx.x]), weight + ea);
                cp_async16_l1(smem_addr(&piece[place][3][threadIdx.x]), weight + eb);
            }
            advance(next_tt, next_at);
        }
        cp_async_commit();
    };
    if (tt < live) {  // on their way while the angles are made
        what(at);
        const __nv_bfloat16 *src = source(tt);
        wa = *reinterpret_cast<const uint4 *>(src + (is_v ? 8 * j : ea));
        wb = *reinterpret_cast<const uint4 *>(src + (is_v ? D / 2 + 8 * j : eb));
        if (const __nv_bfloat16 *weight = weights()) {
            ga = *reinterpret_cast<const uint4 *>(weight + ea);
            gb = *reinterpret_cast<const uint4 *>(weight + eb);
        }
        advance(next_tt, next_at);
    }
#pragma unroll
    for (int i = 0; i < kPieces - 1; ++i) fetch(i);

    for (int x = threadIdx.x; x < live * a.pairs; x += kThreads) {
        const int tok = x / a.pairs, p = x - tok * a.pairs;
        int axis = a.pair_axis ? a.pair_axis[p] : 0;
        if (axis < 0 || axis >= a.num_axes) {
            set_device_error(a.err, PA_DEVERR_BAD_AXIS);
            axis = 0;
        }
        const int pos = a.positions[static_cast<int64_t>(axis) * a.num_tokens + t0 + tok];
        const uint64_t frac = turn_fraction(a.inv_freq[p]);
        const uint64_t phase = frac * static_cast<uint64_t>(static_cast<int64_t>(pos));
        // the upper 32 bits, signed: half turns in [-1, 1)
        const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f;
        float s, c;
        sincospif(half_turns, &s, &c);
        const int to = ADJACENT ? p : spread<D / 2>(p);
        cs[tok][to] = c * a.magnitude;
        sn[tok][to] = s * a.magnitude;
    }
    if constexpr (NORM == kShared)
        for (int x = threadIdx.x; x < 2 * D; x += kThreads) {
            const __nv_bfloat16 *weight = x < D ? a.q_weight : a.k_weight;
            weight_s[x / D][spread<D>(x % D)] = weight ? __bfloat162float(weight[x % D]) + a.weight_offset : 1.f;
        }
    if (threadIdx.x < live) {
        int32_t slot = a.slots[t0 + threadIdx.x];
        if (slot >= a.num_slots) {
            if (blockIdx.y == 0) set_device_error(a.err, PA_DEVERR_BAD_SLOT);
            slot = -1;
        }
        row_s[threadIdx.x] = slot < 0 ? -1 : static_cast<int64_t>(slot / a.block_size) * a.num_kv_heads * a.block_size + slot % a.block_size;
    }
    __syncthreads();

    auto store = [&]() {
        const int64_t t = t0 + tt;
        const int64_t row = row_s[tt];
        if (!is_q && row < 0) return;
        const int da = is_v ? 8 * j : ea, db = is_v ? D / 2 + 8 * j : eb;
        const int64_t dst = (is_q ? t * a.num_q_heads + h : row + h * a.block_size) * D;
        const bool rotate = turn && !is_v;
        if (!rotate && (!FP8 || is_q) && (!NORM || is_v)) {  // bits as they are
            __nv_bfloat16 *to = is_q ? a.q_out : reinterpret_cast<__nv_bfloat16 *>(is_v ? a.v_cache : a.k_cache);
            *reinterpret_cast<uint4 *>(to + dst + da) = wa;
            *reinterpret_cast<uint4 *>(to + dst + db) = wb;
            return;
        }
        float2 xa[4], xb[4];
        unpack8(wa, xa);
        unpack8(wb, xb);
        if constexpr (NORM) {
            if (!is_v) {
                float2 sum = mul2(xa[0], xa[0]), more = mul2(xb[0], xb[0]);
#pragma unroll
                for (int u = 1; u < 4; ++u) {
                    sum = fma2(xa[u], xa[u], sum);
                    more = fma2(xb[u], xb[u], more);
                }
                sum = add2(sum, more);
                float all = sum.x + sum.y;
                const unsigned lanes = ((1u << VPR) - 1u) << (threadIdx.x & 31 & ~(VPR - 1));  // the row's
#pragma unroll
                for (int d = 1; d < VPR; d *= 2) all += __shfl_xor_sync(lanes, all, d);
                const float r = rsqrtf(all * (1.f / D) + a.eps);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    xa[u] = mul2(xa[u], make_float2(r, r));
                    xb[u] = mul2(xb[u], make_float2(r, r));
                }
                float2 g[4];
                auto scale = [&](float2 (&x)[4], int e, const uint4 &raw) {  // elements e .. e + 7
                    if constexpr (NORM == kShared) {
                        take8<D>(weight_s[is_q ? 0 : 1], e / 8, g);
                    } else {
                        if (!(is_q ? a.q_weight : a.k_weight)) return;
                        unpack8(raw, g);
#pragma unroll
                        for (int u = 0; u < 4; ++u) g[u] = add2(g[u], make_float2(a.weight_offset, a.weight_offset));
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) x[u] = mul2(x[u], g[u]);
                };
                scale(xa, ea, ga);
                scale(xb, eb, gb);
            }
        }
        if (rotate) {
            // (p, r) of a pair become (p c - r s, p s + r c): the inner product is rounded,
            // then a fused multiply-add
            auto turn2 = [](float2 &p, float2 &r, float2 co, float2 si) {
                const float2 u = mul2(r, si), w = mul2(r, co), x = p;
                p = fma2(x, co, make_float2(-u.x, -u.y));
                r = fma2(x, si, w);
            };
            if constexpr (ADJACENT) {
                auto turn4 = [&](float2 (&x)[4], int first) {  // by pairs first .. first + 3
                    const float4 c = *reinterpret_cast<const float4 *>(cs[tt] + first), s = *reinterpret_cast<const float4 *>(sn[tt] + first);
#pragma unroll
                    for (int u = 0; u < 4; u += 2) {
                        float2 p = make_float2(x[u].x, x[u + 1].x), r = make_float2(x[u].y, x[u + 1].y);
                        turn2(p, r, u ? make_float2(c.z, c.w) : make_float2(c.x, c.y), u ? make_float2(s.z, s.w) : make_float2(s.x, s.y));
                        x[u] = make_float2(p.x, r.x);
                        x[u + 1] = make_float2(p.y, r.y);
                    }
                };
                turn4(xa, 4 * j);
                if (turn_b) turn4(xb, D / 4 + 4 * j);
            } else {
                float2 c[4], s[4];
                take8<D / 2>(cs[tt], j, c);
                take8<D / 2>(sn[tt], j, s);
#pragma unroll
                for (int u = 0; u < 4; ++u) turn2(xa[u], xb[u], c[u], s[u]);
            }
        }
        // the bits as they are of a vector that nothing is done to
        auto second = [&] { return ADJACENT && !NORM && !turn_b ? wb : pack8(xb); };
        if (is_q) {
            *reinterpret_cast<uint4 *>(a.q_out + dst + da) = pack8(xa);
            *reinterpret_cast<uint4 *>(a.q_out + dst + db) = second();
        } else if constexpr (FP8) {
            const float *scales = is_v ? a.v_scales : a.k_scales;
            const Divisor by = scales ? Divisor::of(scales[h]) : a.kv_scale;
            uint8_t *to = is_v ? a.v_cache : a.k_cache;
            *reinterpret_cast<uint2 *>(to + dst + da) = codes8(xa, by);
            *reinterpret_cast<uint2 *>(to + dst + db) = codes8(xb, by);
        } else {
            __nv_bfloat16 *to = reinterpret_cast<__nv_bfloat16 *>(a.k_cache);
            *reinterpret_cast<uint4 *>(to + dst + da) = pack8(xa);
            *reinterpret_cast<uint4 *>(to + dst + db) = second();
        }
    };
    dependent_release();
    for (int place = 0; tt < live; place = place + 1 == kPieces ? 0 : place + 1) {
        what(at);
        store();
        advance(tt, at);
        if (tt >= live) break;
        cp_async_wait<kPieces - 2>();
        wa = piece[place][0][threadIdx.x];
        wb = piece[place][1][threadIdx.x];
        if constexpr (NORM == kHeads) {
            ga = piece[place][2][threadIdx.x];
            gb = piece[place][3][threadIdx.x];
        }
        fetch(place == 0 ? kPieces - 1 : place - 1);
    }
}

// Grids of several waves want a fifth CTA on each SM at head dim 128 (32 + 8 heads:
// 700 tokens 3.8 against 4.4 us, 8192 32.5 against 33.1), others the registers (1000
// tokens 4.6 against 5.2 us), and so does NORM, which would keep some of its values in
// memory (8192 tokens 34.5 against 36.8 us, E4M3 34.5 against 40.2).
static constexpr bool five_to_an_sm(int head_dim, bool norm, int64_t ctas) { return head_dim == 128 && !norm && ctas > 4 * 152; }

// Tokens to a CTA: the least of tokens on the fullest SM plus, for each wave of
// CTAs, its start (the angles) and its last CTA's own time, in units of 6144
// elements.  Weights fitted to tiles of 1 to 8 over 256 to 8192 tokens of 48 and
// 80 rows at both head dims, with and without NORM: 0.6% from the best tile on average,
// 7% at worst.  (32 + 8 heads, 700 tokens: 3.9 us with 1 to a CTA, 5.1 with 4; 3500: 15.7
// with 5, 19.5 with 1; NORM, 2500: 13.5 with 5, 15.2 with 4.)
static int tokens_per_cta(int num_tokens, int rows, int head_dim, bool norm) {
    const double work = static_cast<double>(rows) * head_dim / 6144;
    int best = 1;
    double least = INFINITY;
    for (int tile = 1; tile <= kMaxTile; ++tile) {
        const int64_t ctas = (static_cast<int64_t>(num_tokens) + tile - 1) / tile;
        const int64_t places = static_cast<int64_t>(five_to_an_sm(head_dim, norm, ctas) ? 5 : 4) * 152;
        const int64_t waves = (ctas + places - 1) / places, fullest = (ctas + 151) / 152 * tile;
        const double cost = work * fullest + waves * (4.25 + 2 * work * tile);
        if (cost < least) {
            least = cost;
            best = tile;
        }
    }
    return best;
}

template <int D, bool FP8, bool ADJACENT, int NORM>
static cudaError_t launch_ctas(const Args &a, dim3 grid, cudaStream_t stream) {
    if constexpr (D == 128 && NORM == kNone)
        if (five_to_an_sm(D, false, static_cast<int64_t>(grid.x) * grid.y))
            return launch_dependent(append_kernel<D, FP8, ADJACENT, NORM, 5>, grid, kThreads, 0, 0, stream, a);
    return launch_dependent(append_kernel<D, FP8, ADJACENT, NORM, 4>, grid, kThreads, 0, 0, stream, a);
}

template <int D, bool FP8, int NORM>
static cudaError_t launch_adjacent(const Args &a, bool adjacent, dim3 grid, cudaStream_t stream) {
    return adjacent ? launch_ctas<D, FP8, true, NORM>(a, grid, stream) : launch_ctas<D, FP8, false, NORM>(a, grid, stream);
}

template <int D, bool FP8>
static cudaError_t launch(const Args &a, bool adjacent, int norm, dim3 grid, cudaStream_t stream) {
    return norm == kNone     ? launch_adjacent<D, FP8, kNone>(a, adjacent, grid, stream)
           : norm == kShared ? launch_adjacent<D, FP8, kShared>(a, adjacent, grid, stream)
                             : launch_adjacent<D, FP8, kHeads>(a, adjacent, grid, stream);
}

// What the norm adds to a call.
struct Norm {
    const void *q_weight;
    int64_t q_weight_stride;
    const void *k_weight;
    int64_t k_weight_stride;
    float weight_offset, eps;
};

// `norm`: null without one.
static pa_status append(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                        const Norm *norm, const int32_t *positions, int num_axes, const double *inv_freq,
                        const int32_t *pair_axis, int rotary_dim, int adjacent, float magnitude,
                        const int32_t *slot_mapping, int num_tokens, int num_q_heads, void *q_out, void *k_cache,
                        void *v_cache, int num_blocks, int num_kv_heads, int head_dim, int block_size,
                        pa_kv_dtype kv_dtype, float kv_scale, const float *k_scales, const float *v_scales,
                        cudaStream_t stream) {
    clear_error();
    if (num_tokens < 0 || num_q_heads < 0 || num_kv_heads <= 0 || num_blocks <= 0)
        return fail(PA_ERR_INVALID_ARG, "bad size (num_tokens=%d, num_q_heads=%d, num_kv_heads=%d, num_blocks=%d)",
                    num_tokens, num_q_heads, num_kv_heads, num_blocks);
    if (num_q_heads > 65535 || num_kv_heads > 65535)
        return fail(PA_ERR_UNSUPPORTED, "more than 65535 heads");
    if (head_dim != 64 && head_dim != 128)
        return fail(PA_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", head_dim);
    if (block_size != 16 && block_size != 32)
        return fail(PA_ERR_UNSUPPORTED, "block_size %d (supported: 16, 32)", block_size);
    if (kv_dtype != PA_KV_BF16 && kv_dtype != PA_KV_FP8_E4M3)
        return fail(PA_ERR_UNSUPPORTED, "kv_dtype %d", static_cast<int>(kv_dtype));
    if (rotary_dim <= 0 || rotary_dim > head_dim)
        return fail(PA_ERR_INVALID_ARG, "rotary_dim %d outside 1..head_dim %d", rotary_dim, head_dim);
    if (rotary_dim % 16 != 0)
        return fail(PA_ERR_UNSUPPORTED, "rotary_dim %d is not a multiple of 16", rotary_dim);
    if (num_axes < 1 || num_axes > 16)
        return fail(num_axes < 1 ? PA_ERR_INVALID_ARG : PA_ERR_UNSUPPORTED, "num_axes %d (supported: 1..16)", num_axes);
    if (num_axes > 1 && !pair_axis)
        return fail(PA_ERR_INVALID_ARG, "pair_axis is needed with more than one axis");
    if (!(magnitude > 0.f && magnitude <= 3.4e38f))
        return fail(PA_ERR_INVALID_ARG, "magnitude must be positive and finite");
    if ((k_scales == nullptr) != (v_scales == nullptr))
        return fail(PA_ERR_INVALID_ARG, "k_scales and v_scales must both be given or both be NULL");
    if (k_scales && kv_dtype != PA_KV_FP8_E4M3)
        return fail(PA_ERR_INVALID_ARG, "per-head scales need an E4M3 cache");
    if (kv_dtype == PA_KV_FP8_E4M3 && !k_scales && !(kv_scale > 0.f && kv_scale <= 3.4e38f))
        return fail(PA_ERR_INVALID_ARG, "fp8 kv_scale must be positive and finite");
    if (static_cast<int64_t>(num_blocks) * block_size > 0x7fffffffLL)
        return fail(PA_ERR_UNSUPPORTED, "pool of %d blocks exceeds 2^31 slots", num_blocks);
    if (norm) {
        if (!(norm->eps >= 1e-12f && norm->eps <= 3.4e38f))
            return fail(PA_ERR_INVALID_ARG, "eps must be finite and at least 1e-12");
        if (!(norm->weight_offset >= -3.4e38f && norm->weight_offset <= 3.4e38f))
            return fail(PA_ERR_INVALID_ARG, "weight_offset must be finite");
        for (const auto &[weight, stride, heads] : {std::tuple(norm->q_weight, norm->q_weight_stride, num_q_heads),
                                                    std::tuple(norm->k_weight, norm->k_weight_stride, num_kv_heads)}) {
            if (!weight) continue;
            if (!aligned16(weight)) return fail(PA_ERR_INVALID_ARG, "weights must be 16-byte aligned");
            if (stride % 8 || stride < 0 || (stride && heads > 1 && stride < head_dim))
                return fail(PA_ERR_INVALID_ARG, "a weight stride is 0, or a multiple of 8 elements and at least head_dim");
        }
    }
    if (num_tokens == 0) return PA_OK;
    if (!k || !v || !positions || !inv_freq || !slot_mapping || !k_cache || !v_cache ||
        (num_q_heads > 0 && (!q || !q_out)))
        return fail(PA_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
        (num_q_heads > 0 && (!aligned16(q) || !aligned16(q_out))))
        return fail(PA_ERR_INVALID_ARG, "q, k, v, q_out, k_cache and v_cache must be 16-byte aligned");
    const int64_t qrow = static_cast<int64_t>(num_q_heads) * head_dim;
    const int64_t krow = static_cast<int64_t>(num_kv_heads) * head_dim;
    if (k_stride % 8 || v_stride % 8 || (num_q_heads > 0 && q_stride % 8))
        return fail(PA_ERR_INVALID_ARG, "token strides must be multiples of 8 elements");
    if (num_tokens > 1 && (k_stride < krow || v_stride < krow || (num_q_heads > 0 && q_stride < qrow)))
        return fail(PA_ERR_INVALID_ARG, "a token stride is smaller than one token's rows");
    if (num_q_heads > 0 && !(q == q_out && (num_tokens == 1 || q_stride == qrow))) {
        const size_t span = (static_cast<size_t>(num_tokens - 1) * q_stride + qrow) * 2;
        if (overlaps(q, span, q_out, static_cast<size_t>(num_tokens) * qrow * 2))
            return fail(PA_ERR_INVALID_ARG, "q_out overlaps q but is not q itself");
    }
    for (const auto &[rows, stride] : {std::pair(k, k_stride), std::pair(v, v_stride)}) {
        const size_t span = (static_cast<size_t>(num_tokens - 1) * stride + krow) * 2;
        if (num_q_heads > 0 && overlaps(rows, span, q_out, static_cast<size_t>(num_tokens) * qrow * 2))
            return fail(PA_ERR_INVALID_ARG, "q_out overlaps k or v");
    }
    if (norm && num_q_heads > 0)
        for (const auto &[weight, stride, heads] : {std::tuple(norm->q_weight, norm->q_weight_stride, num_q_heads),
                                                    std::tuple(norm->k_weight, norm->k_weight_stride, num_kv_heads)}) {
            const size_t span = (static_cast<size_t>(heads - 1) * stride + head_dim) * 2;
            if (weight && overlaps(weight, span, q_out, static_cast<size_t>(num_tokens) * qrow * 2))
                return fail(PA_ERR_INVALID_ARG, "q_out overlaps the weights");
        }
    unsigned int *err = device_error_word();
    if (!err) return fail(PA_ERR_CUDA, "cannot resolve the device error word");

    Args a;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.v = static_cast<const __nv_bfloat16 *>(v);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.pair_axis = pair_axis;
    a.slots = slot_mapping;
    a.q_out = static_cast<__nv_bfloat16 *>(q_out);
    a.k_cache = static_cast<uint8_t *>(k_cache);
    a.v_cache = static_cast<uint8_t *>(v_cache);
    a.num_slots = static_cast<int64_t>(num_blocks) * block_size;
    a.num_tokens = num_tokens;
    a.num_axes = num_axes;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.block_size = block_size;
    a.pairs = rotary_dim / 2;
    a.magnitude = magnitude;
    a.kv_scale = Divisor::of(kv_scale);
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.err = err;
    a.q_weight = norm ? static_cast<const __nv_bfloat16 *>(norm->q_weight) : nullptr;
    a.k_weight = norm ? static_cast<const __nv_bfloat16 *>(norm->k_weight) : nullptr;
    a.q_weight_stride = a.q_weight ? norm->q_weight_stride : 0;
    a.k_weight_stride = a.k_weight ? norm->k_weight_stride : 0;
    a.weight_offset = norm ? norm->weight_offset : 0.f;
    a.eps = norm ? norm->eps : 0.f;
    const int kind = !norm ? kNone : a.q_weight_stride || a.k_weight_stride ? kHeads : kShared;
    const int rows = num_q_heads + 2 * num_kv_heads;
    a.tile = tokens_per_cta(num_tokens, rows, head_dim, norm != nullptr);
    const int at_once = kThreads / (head_dim / 16);  // rows of one pass of the CTA's threads
    // With few tokens a token's rows are shared out too, up to four CTAs to an SM.
    const int shares = std::max(1, std::min((rows + at_once - 1) / at_once, 4 * 152 / num_tokens));
    a.rows_per_y = (rows + shares - 1) / shares;
    const dim3 grid((static_cast<unsigned>(num_tokens) + a.tile - 1) / a.tile, (rows + a.rows_per_y - 1) / a.rows_per_y);
    const bool fp8 = kv_dtype == PA_KV_FP8_E4M3, adj = adjacent != 0;
    const cudaError_t e = head_dim == 128 ? (fp8 ? launch<128, true>(a, adj, kind, grid, stream)
                                                 : launch<128, false>(a, adj, kind, grid, stream))
                                          : (fp8 ? launch<64, true>(a, adj, kind, grid, stream)
                                                 : launch<64, false>(a, adj, kind, grid, stream));
    return cuda_check(e, "rope append launch");
}

}  // namespace rope
}  // namespace pa

using namespace pa;

extern "C" {

pa_status pa_rope_append(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                         int64_t v_stride, const int32_t *positions, int num_axes, const double *inv_freq,
                         const int32_t *pair_axis, int rotary_dim, int adjacent, float magnitude,
                         const int32_t *slot_mapping, int num_tokens, int num_q_heads, void *q_out, void *k_cache,
                         void *v_cache, int num_blocks, int num_kv_heads, int head_dim, int block_size,
                         pa_kv_dtype kv_dtype, float kv_scale, const float *k_scales, const float *v_scales,
                         cudaStream_t stream) {
    return rope::append(q, q_stride, k, k_stride, v, v_stride, nullptr, positions, num_axes, inv_freq, pair_axis,
                        rotary_dim, adjacent, magnitude, slot_mapping, num_tokens, num_q_heads, q_out, k_cache, v_cache,
                        num_blocks, num_kv_heads, head_dim, block_size, kv_dtype, kv_scale, k_scales, v_scales, stream);
}

pa_status pa_norm_rope_append(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                              int64_t v_stride, const void *q_weight, int64_t q_weight_stride, const void *k_weight,
                              int64_t k_weight_stride, float weight_offset, float eps, const int32_t *positions,
                              int num_axes, const double *inv_freq, const int32_t *pair_axis, int rotary_dim,
                              int adjacent, float magnitude, const int32_t *slot_mapping, int num_tokens,
                              int num_q_heads, void *q_out, void *k_cache, void *v_cache, int num_blocks,
                              int num_kv_heads, int head_dim, int block_size, pa_kv_dtype kv_dtype, float kv_scale,
                              const float *k_scales, const float *v_scales, cudaStream_t stream) {
    const rope::Norm norm{q_weight, q_weight_stride, k_weight, k_weight_stride, weight_offset, eps};
    return rope::append(q, q_stride, k, k_stride, v, v_stride, &norm, positions, num_axes, inv_freq, pair_axis,
                        rotary_dim, adjacent, magnitude, slot_mapping, num_tokens, num_q_heads, q_out, k_cache, v_cache,
                        num_blocks, num_kv_heads, head_dim, block_size, kv_dtype, kv_scale, k_scales, v_scales, stream);
}

}  // extern "C"
