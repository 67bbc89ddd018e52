// Rotate-and-append: the position rotation of a batch of new tokens' q and k
// rows, and the write of their k and v rows into the paged cache, in one
// kernel ("Optimizing Llama 3.1 405B Inference with vLLM PagedAttention",
// section "PagedAttention Mechanics": a token's K and V are appended on
// arrival; the pages leave the rotation to the model).
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
// Bound: memory.  Every q, k, v element is read once and written once: 8192
// tokens of 32 query and 8 KV heads, 201 MB, take 35 us, where a library copy of
// as much takes 32.5; few tokens are bound by the launch (one: 2.0 us) and by the
// chain position, sine and cosine, row, so a thread's first row is on its way
// while the angles are made.
#include <algorithm>
#include <cstring>
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
// code is 0 or the largest, whatever the last place.  (8192 tokens, 32 + 8 heads:
// 36.5 us with it, 39.5 with a division for every element; 256 tokens of 64 + 8
// heads 3.7 and 4.0.)
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
};

constexpr int kThreads = 256;
constexpr int kMaxTile = 8;

__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8]) {
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(h[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack2<false>(x[0], x[1]), pack2<false>(x[2], x[3]), pack2<false>(x[4], x[5]),
                      pack2<false>(x[6], x[7]));
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
__device__ __forceinline__ uint2 codes8(const float (&x)[8], const Divisor &by) {
    uint32_t w[2] = {0, 0};
    uint32_t least = 0xffffffffu;  // of the endings, plus 4, in the upper 19 bits
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 y = make_float2(__fmul_rn(x[i], by.inverse), __fmul_rn(x[i + 1], by.inverse));
        least = min(least, min(__float_as_uint(y.x) * 8192u + 32768u, __float_as_uint(y.y) * 8192u + 32768u));
        w[i / 4] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3)) << 8 * (i % 4);
    }
    if (least < by.near) {
        w[0] = w[1] = 0;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float2 y = make_float2(__fdiv_rn(x[i], by.scale), __fdiv_rn(x[i + 1], by.scale));
            w[i / 4] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3)) << 8 * (i % 4);
        }
    }
    return make_uint2(w[0], w[1]);
}

// A thread works on 16 elements of one head's row at a time: with pairs
// (i, i + R/2) elements 8j .. 8j+7 and their partners, with adjacent pairs
// elements 16j .. 16j+15; either way pairs 8j .. 8j+7, and two 16-byte loads.
// Its j is the same for every row it takes.
// CTAS: of the kernel to an SM, which caps its registers.
template <int D, bool FP8, bool ADJACENT, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS) append_kernel(const Args a) {
    constexpr int VPR = D / 16;  // threads to a row
    __shared__ __align__(16) float cs[kMaxTile][D / 2], sn[kMaxTile][D / 2];
    __shared__ int64_t row_s[kMaxTile];  // the slot's row of head 0, or -1
    dependent_wait();
    const int t0 = blockIdx.x * a.tile;
    const int live = min(a.tile, a.num_tokens - t0);
    const int j = threadIdx.x % VPR;
    const int rows = a.num_q_heads + 2 * a.num_kv_heads;
    const int row0 = blockIdx.y * a.rows_per_y;
    const int nrows = min(a.rows_per_y, rows - row0);
    const bool turn = 8 * j < a.pairs;
    // first elements of the thread's two vectors
    const int rest = 2 * a.pairs + 16 * (j - a.pairs / 8);
    const int ea = !turn ? rest : ADJACENT ? 16 * j : 8 * j;
    const int eb = !turn || ADJACENT ? ea + 8 : a.pairs + 8 * j;
    uint4 wa, wb;  // the thread's present piece
    const int first = threadIdx.x / VPR;
    int tt = first / nrows, at = first - tt * nrows;  // token and row of the piece
    int h;
    bool is_q, is_v;
    auto load = [&]() {
        const int row = row0 + at;
        const int64_t t = t0 + tt;
        is_q = row < a.num_q_heads;
        is_v = row >= a.num_q_heads + a.num_kv_heads;
        h = row - (is_q ? 0 : is_v ? a.num_q_heads + a.num_kv_heads : a.num_q_heads);
        const __nv_bfloat16 *src = (is_q ? a.q + t * a.q_stride : is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride) +
                                   static_cast<int64_t>(h) * D;
        wa = *reinterpret_cast<const uint4 *>(src + (is_v ? 16 * j : ea));
        wb = *reinterpret_cast<const uint4 *>(src + (is_v ? 16 * j + 8 : eb));
    };
    if (tt < live) load();  // on its way while the angles are made

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
        cs[tok][p] = c * a.magnitude;
        sn[tok][p] = s * a.magnitude;
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
        const int da = is_v ? 16 * j : ea, db = is_v ? da + 8 : eb;
        const int64_t dst = (is_q ? t * a.num_q_heads + h : row + h * a.block_size) * D;
        const bool rotate = turn && !is_v;
        if (!rotate && (!FP8 || is_q)) {  // bits as they are
            __nv_bfloat16 *to = is_q ? a.q_out : reinterpret_cast<__nv_bfloat16 *>(is_v ? a.v_cache : a.k_cache);
            *reinterpret_cast<uint4 *>(to + dst + da) = wa;
            *reinterpret_cast<uint4 *>(to + dst + db) = wb;
            return;
        }
        float xa[8], xb[8];
        unpack8(wa, xa);
        unpack8(wb, xb);
        if (rotate) {
            float c[8], s[8];
#pragma unroll
            for (int u = 0; u < 8; u += 4) {
                *reinterpret_cast<float4 *>(c + u) = *reinterpret_cast<const float4 *>(&cs[tt][8 * j + u]);
                *reinterpret_cast<float4 *>(s + u) = *reinterpret_cast<const float4 *>(&sn[tt][8 * j + u]);
            }
            auto rot = [&](float &u, float &w, int i8) {
                const float p = u, r = w;
                u = fmaf(p, c[i8], -(r * s[i8]));
                w = fmaf(p, s[i8], r * c[i8]);
            };
            if constexpr (ADJACENT) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    rot(xa[2 * u], xa[2 * u + 1], u);
                    rot(xb[2 * u], xb[2 * u + 1], 4 + u);
                }
            } else {
#pragma unroll
                for (int u = 0; u < 8; ++u) rot(xa[u], xb[u], u);
            }
        }
        if (is_q) {
            *reinterpret_cast<uint4 *>(a.q_out + dst + da) = pack8(xa);
            *reinterpret_cast<uint4 *>(a.q_out + dst + db) = pack8(xb);
        } else if constexpr (FP8) {
            const float *scales = is_v ? a.v_scales : a.k_scales;
            const Divisor by = scales ? Divisor::of(scales[h]) : a.kv_scale;
            uint8_t *to = is_v ? a.v_cache : a.k_cache;
            *reinterpret_cast<uint2 *>(to + dst + da) = codes8(xa, by);
            *reinterpret_cast<uint2 *>(to + dst + db) = codes8(xb, by);
        } else {
            __nv_bfloat16 *to = reinterpret_cast<__nv_bfloat16 *>(a.k_cache);
            *reinterpret_cast<uint4 *>(to + dst + da) = pack8(xa);
            *reinterpret_cast<uint4 *>(to + dst + db) = pack8(xb);
        }
    };
    dependent_release();
    while (tt < live) {
        store();
        for (at += kThreads / VPR; at >= nrows; at -= nrows) ++tt;
        if (tt < live) load();
    }
}

// Grids of several waves want a fifth CTA on each SM at head dim 128 (8192
// tokens, 32 + 8 heads: 34.8 against 38.9 us, E4M3 36.5 against 38.8), others the
// registers (1000 tokens 5.6 against 6.4 us; 8192 of head dim 64, E4M3 cache, 21.1
// against 22.6).
static constexpr bool five_to_an_sm(int head_dim, int64_t ctas) { return head_dim == 128 && ctas > 4 * 152; }

// Tokens to a CTA: the least of tokens on the fullest SM plus, for each wave of
// CTAs, its start (the angles) and its last CTA's own time, in units of 6144
// elements.  Weights fitted to tiles of 1 to 8 over 400 to 7000 tokens of 24 to
// 80 rows at both head dims: within 2% of the best tile.  (32 + 8 heads, 700
// tokens: 4.3 us with 1 to a CTA, 5.3 with 2; 1500: 6.4 with 2, 8.5 with 4; 3500:
// 16.8 with 5, 19.4 with 4; 8192: 34.7 with 6, 39.6 with 8.)
static int tokens_per_cta(int num_tokens, int rows, int head_dim) {
    const double work = static_cast<double>(rows) * head_dim / 6144;
    int best = 1;
    double least = INFINITY;
    for (int tile = 1; tile <= kMaxTile; ++tile) {
        const int64_t ctas = (static_cast<int64_t>(num_tokens) + tile - 1) / tile;
        const int64_t places = static_cast<int64_t>(five_to_an_sm(head_dim, ctas) ? 5 : 4) * 152;
        const int64_t waves = (ctas + places - 1) / places, fullest = (ctas + 151) / 152 * tile;
        const double cost = work * fullest + waves * (3.5 + 1.5 * work * tile);
        if (cost < least) {
            least = cost;
            best = tile;
        }
    }
    return best;
}

template <int D, bool FP8, bool ADJACENT>
static cudaError_t launch_ctas(const Args &a, dim3 grid, cudaStream_t stream) {
    if constexpr (D == 128)
        if (five_to_an_sm(D, static_cast<int64_t>(grid.x) * grid.y))
            return launch_dependent(append_kernel<D, FP8, ADJACENT, 5>, grid, kThreads, 0, 0, stream, a);
    return launch_dependent(append_kernel<D, FP8, ADJACENT, 4>, grid, kThreads, 0, 0, stream, a);
}

template <int D, bool FP8>
static cudaError_t launch(const Args &a, bool adjacent, dim3 grid, cudaStream_t stream) {
    return adjacent ? launch_ctas<D, FP8, true>(a, grid, stream) : launch_ctas<D, FP8, false>(a, grid, stream);
}

}  // namespace rope
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_rope_append(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                    const void *v, int64_t v_stride, const int32_t *positions,
                                    int num_axes, const double *inv_freq, const int32_t *pair_axis,
                                    int rotary_dim, int adjacent, float magnitude,
                                    const int32_t *slot_mapping, int num_tokens, int num_q_heads,
                                    void *q_out, void *k_cache, void *v_cache, int num_blocks,
                                    int num_kv_heads, int head_dim, int block_size,
                                    pa_kv_dtype kv_dtype, float kv_scale, const float *k_scales,
                                    const float *v_scales, cudaStream_t stream) {
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
    unsigned int *err = device_error_word();
    if (!err) return fail(PA_ERR_CUDA, "cannot resolve the device error word");

    rope::Args a;
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
    a.kv_scale = rope::Divisor::of(kv_scale);
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.err = err;
    const int rows = num_q_heads + 2 * num_kv_heads;
    a.tile = rope::tokens_per_cta(num_tokens, rows, head_dim);
    const int at_once = rope::kThreads / (head_dim / 16);  // rows of one pass of the CTA's threads
    // With few tokens a token's rows are shared out too, up to four CTAs to an SM.
    const int shares = std::max(1, std::min((rows + at_once - 1) / at_once, 4 * 152 / num_tokens));
    a.rows_per_y = (rows + shares - 1) / shares;
    const dim3 grid((static_cast<unsigned>(num_tokens) + a.tile - 1) / a.tile, (rows + a.rows_per_y - 1) / a.rows_per_y);
    const bool fp8 = kv_dtype == PA_KV_FP8_E4M3, adj = adjacent != 0;
    const cudaError_t e = head_dim == 128 ? (fp8 ? rope::launch<128, true>(a, adj, grid, stream)
                                                 : rope::launch<128, false>(a, adj, grid, stream))
                                          : (fp8 ? rope::launch<64, true>(a, adj, grid, stream)
                                                 : rope::launch<64, false>(a, adj, grid, stream));
    return cuda_check(e, "rope append launch");
}
