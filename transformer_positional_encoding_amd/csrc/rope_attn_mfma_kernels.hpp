// rope_attn_mfma_kernels.hpp -- attention over a cache held in 4 bits on the
// matrix cores: 16-bit queries, rows of whole 8-lane chunks up to 256 lanes,
// one scale a row or groups of whole 16 lanes.
// Included by the rope_attn_*.hip files of a type each.
//
// A wave takes 16 query rows (NT such tiles) and 64 cached tokens at a time.
// Both products have the cached rows as their first operand, so that a query
// row is a column of every accumulator, one lane's: x^T = K Q^T, o^T = V^T P^T.
// The weights then leave the first product in the very lanes and order in which
// the second takes them (a product's sum may take its tokens in any order), and
// a row's running maximum and sum are a lane's own but for two exchanges.
//
// Codes to numbers. A nibble n = code + 8 put into the fraction of 16 makes 16 +
// n, an exact bf16 and fp16 number, for a shift and one more operation per two
// codes; K stays like that and the accumulator starts from -24 sum(q). V's
// sums run over many tokens, where such a part would cost digits: its nibbles
// become 1024 + n in fp16 and lose the 1032 by a packed subtraction. The order
// of lanes within a product is free too: a lane takes a 32-bit word of 8 codes
// of a K row as it comes (pairs of nibbles 16 bits apart, q's fragment in the
// same order), and of V the words of 8 tokens at the same place of their rows,
// whose 16-bit halves, put side by side, hold the codes of two tokens at equal
// nibbles. With a scale for each segment of 32 lanes (VF) a segment has to be
// whole products, a byte a lane: lanes in fours exchange the bytes of words of
// four segments. With one for each half of a segment, each half has a product of
// its own, the other half's lanes of q, or of V, being 0.
//
// Scales stay outside of the products: K's multiply the finished sums of their
// lanes (one a row, or one for each 32-lane step, KF), V's the weights. exp(x -
// m) times V's scale is rounded to fp16 (2^-11 of it, where bf16's store rounds
// by 2^-8 afterwards), times a power of two, 2^-e. e is set from the row's
// largest such weight of the scale's lanes when m moves or a tile's scales could
// take a weight past 2^15; between that the weights are at most 2^6 * 2^9 of
// what e was set from, and what is below 2^-14 loses digits, at most 2^-25. m
// follows the maximum when it is passed by 2^6; a tile that moves neither m nor
// e leaves the accumulators as they are.
//
// The bytes are 4 bits a code; at the rate of a large copy that is 10^13 codes a
// second, against 4 * 10^13 operations of the vector units, so operations per
// code decide: of 64 tokens of 128 lanes, 16384 codes, a wave issues about 680
// (128 for K's numbers, 190 for V's, 230 for 16 rows' softmax, the rest for
// addresses), 1120 with a scale for 32 lanes, 760 and 1600 with 32 rows.
//
// Three kernels differ in where a tile's numbers come from:
//   rope_attn_mfma_kernel    any heads, strides and pages: loads go straight to
//       registers, a tile ahead. Four waves of a block take heads beside each
//       other, or share the rows and take tiles in turn (joined in LDS), or have
//       rows of their own.
//   rope_attn_heads_kernel   up to 64 rows, four heads that lie together.
//   rope_attn_shared_kernel  more rows of one head.
#pragma once

#include "rope_attn_kernels.hpp"
#include "rope_dma.hpp"

namespace rope {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t v3u __attribute__((ext_vector_type(3)));

struct AttnVecArgs : AttnArgs {
    // what a block's four waves have of their own: cached heads, turns at the
    // tokens (whose results are joined), tiles of rows; one times another is 4
    uint32_t head_waves, token_waves, row_waves;
    uint32_t k_groups, v_groups;   // scales of a row
    uint32_t k_group, v_group;     // lanes of each
};

template <int DT>
__device__ __forceinline__ f32x4 attn_mfma(const v4u& a, const v4u& b, const f32x4& c)
{
    if constexpr (DT == ROPE_DTYPE_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Constants in a register of each lane, or one of the wave: one of either takes
// part in three-operand logic as two literals could not.
__device__ __forceinline__ uint32_t vector_constant(uint32_t v)
{
    uint32_t r;
    asm("v_mov_b32 %0, %1" : "=v"(r) : "i"(v));
    return r;
}

__device__ __forceinline__ uint32_t scalar_constant(uint32_t v)
{
    uint32_t r;
    asm("s_mov_b32 %0, %1" : "=s"(r) : "i"(v));
    return r;
}

// What makes numbers of nibbles: their bits, and what they are added to, with
// the nibbles' upper bit (which turns -8..7 in two's complement into 0..15).
struct Numbers {
    uint32_t mask, one;
};
__device__ __forceinline__ uint32_t number(uint32_t w, const Numbers& c) { return (w & c.mask) ^ c.one; }

// 8 codes as 16 + (code + 8), nibbles i and i + 4 in the halves of word i.
template <int DT>
__device__ __forceinline__ Numbers k_constants()
{
    if constexpr (DT == ROPE_DTYPE_BF16) return Numbers{scalar_constant(0x00780078u), vector_constant(0x41C041C0u)};
    else return Numbers{scalar_constant(0x03C003C0u), vector_constant(0x4E004E00u)};
}

template <int DT>
__device__ __forceinline__ v4u k_numbers(uint32_t w, const Numbers& c)
{
    if constexpr (DT == ROPE_DTYPE_BF16) return v4u{number(w << 3, c), number(w >> 1, c), number(w >> 5, c), number(w >> 9, c)};
    else return v4u{number(w << 6, c), number(w << 2, c), number(w >> 2, c), number(w >> 6, c)};
}

// What makes codes in fp16 of nibbles 0 (1024 + n, less 1032) and 1 (1024 + 16
// n, times 1/16, less 72) of both halves of a word.
struct VConstants {
    Numbers low, high;
};
__device__ __forceinline__ VConstants v_constants()
{
    return VConstants{{scalar_constant(0x000F000Fu), vector_constant(0x64086408u)},
                      {scalar_constant(0x00F000F0u), vector_constant(0x64806480u)}};
}

// The codes at nibble i of both halves of w.
template <int I>
__device__ __forceinline__ uint32_t v_numbers(uint32_t w, const VConstants& c)
{
    w >>= 8 * (I / 2);
    if constexpr (I % 2 == 0) {
        const f16x2 n = __builtin_bit_cast(f16x2, number(w, c.low));
        return __builtin_bit_cast(uint32_t, n - (_Float16)1032.0f);
    } else {
        const f16x2 n = __builtin_bit_cast(f16x2, number(w, c.high)), k{(_Float16)0.0625f, (_Float16)0.0625f},
                    o{(_Float16)-72.0f, (_Float16)-72.0f};
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(n, k, o));
    }
}

// 8 elements of a query row in the order of k_numbers.
__device__ __forceinline__ v4u q_order(const v4u& v)
{
    return v4u{__builtin_amdgcn_perm(v[2], v[0], 0x05040100), __builtin_amdgcn_perm(v[2], v[0], 0x07060302),
               __builtin_amdgcn_perm(v[3], v[1], 0x05040100), __builtin_amdgcn_perm(v[3], v[1], 0x07060302)};
}

// Word i of lane i of four (by lane number) receives byte a of lane a's word in
// its byte a.
__device__ __forceinline__ uint32_t quad_bytes(uint32_t w, uint32_t sel1, uint32_t sel2)
{
    const uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)w, 0xB1, 0xF, 0xF, true);     // lane ^ 1
    w = __builtin_amdgcn_perm(o, w, sel1);
    const uint32_t p = (uint32_t)__builtin_amdgcn_mov_dpp((int)w, 0x4E, 0xF, 0xF, true);     // lane ^ 2
    return __builtin_amdgcn_perm(p, w, sel2);
}

// The largest of three numbers that arithmetic has made (the compiler would first
// quiet each; NaN loses here as there).
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
__device__ __forceinline__ float max3_abs(float a, float b, float c)       // of a and two magnitudes
{
    float r;
    asm("v_max3_f32 %0, %1, |%2|, |%3|" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// The least of 16 lanes' numbers.
__device__ __forceinline__ int32_t least16(int32_t v)
{
    v = min(v, __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true));
    v = min(v, __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true));
    v = min(v, __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true));
    return min(v, __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true));
}

__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Over the four lanes that hold a column: rows of 16 lanes, then halves of the
// wave, change places between two copies.
__device__ __forceinline__ float column_max(float v)
{
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float column_sum(float v)
{
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Scales that a kernel takes of a row: one (0), one for 32 lanes (1) or for 16
// (2, whose segments of 32 are two halves).
constexpr int kHalves = 2;
constexpr int attn_group(int f) { return f == kHalves ? 16 : 32; }
constexpr int attn_groups(int f, int lanes) { return f == 0 ? 1 : lanes / attn_group(f); }

template <int DP, int DVP, int KF, int VF, int NT>
struct alignas(16) AttnLds {
    static constexpr int NGK = attn_groups(KF, DP), NGV = attn_groups(VF, DVP);
    struct Wave {
        int64_t k_at[64], v_at[64];
        float ks[NGK][64], vs[NGV][64];
    };
    struct Join {
        float o[4][16][DVP + 4];
        float m[4][16], l[4][16];
    };
    union {
        Wave wave[4];
        Join join;
    };
};

// A wave's query rows, 16 to a tile, and what it holds of their attention: all
// that does not depend on where a tile's numbers come from.
template <int DT, int DP, int DVP, int KF, int VF, int NT>
struct AttnRows {
    static constexpr int KW = DP / 32;             // steps of a product with K
    static constexpr int VT = DVP / 16;            // products of 16 lanes of V
    static constexpr int NGK = attn_groups(KF, DP), NGV = attn_groups(VF, DVP);
    static constexpr int HK = KF == kHalves ? 2 : 1, HV = VF == kHalves ? 2 : 1;   // scales of a segment

    v4u q[NT][KW * HK];                            // (halves: a step's with the other half's lanes 0)
    float start[NT][NGK];                          // -24 sum(q)
    int32_t last[NT];                              // the last token that a row sees
    f32x4 acc[NT][VT];
    float m[NT], less[NT], l[NT], top[NT][NGV];    // less: m, or 0 where there is none yet
    int32_t e[NT][NGV];
    float safe[NGV];                               // scales that no row's weights outgrow fp16 with

    // Rows r0 to live - 1 (or fewer) of a cached head: a column a row, 8 elements
    // a step in k_numbers' order.
    __device__ __forceinline__ void load(const AttnArgs& a, const AttnSeq& seq, uint32_t b, uint32_t head, uint32_t r0, uint32_t live,
                                         uint32_t n16, uint32_t kq)
    {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint32_t r = min(r0 + t * 16 + n16, live - 1);
            const uint32_t s = fast_div(r, a.rep_div), h = head * a.rep + (r - s * a.rep);
            last[t] = a.causal ? (int32_t)(seq.first + s) : INT32_MAX;
            const gchar* row = as_global(a.q.data) + (b * a.q.sb + s * a.q.ss + h * a.q.sn) * 2;
            float sum = 0.0f;
#pragma unroll
            for (int st = 0; st < KW; ++st) {
                const uint32_t d = KF ? 32 * st + 8 * kq : kq * (DP / 4) + 8 * st;
                v4u v{0, 0, 0, 0};
                if (d < a.D) v = gload<v4u>(row + d * 2);
#pragma unroll
                for (int half = 0; half < HK; ++half) {
                    const v4u part = HK == 1 || (half == 0) == (kq < 2) ? v : v4u{0, 0, 0, 0};
                    Lanes<DT> f;
                    f.unpack(part);
#pragma unroll
                    for (int k = 0; k < 8; ++k) sum += f.v[k];
                    q[t][st * HK + half] = q_order(part);
                    if (KF || st == KW - 1) {
                        start[t][KF ? st * HK + half : 0] = -24.0f * column_sum(sum);
                        sum = 0.0f;
                    }
                }
            }
#pragma unroll
            for (int g = 0; g < NGV; ++g) safe[g] = 0.0f;
            m[t] = kAttnNone;
            less[t] = l[t] = 0.0f;
#pragma unroll
            for (int g = 0; g < NGV; ++g) {
                top[t][g] = 0.0f;
                e[t][g] = 0;
            }
#pragma unroll
            for (int i = 0; i < VT; ++i) acc[t][i] = f32x4{0, 0, 0, 0};
        }
    }

    // x^T = K Q^T, a token a row of the product, less the row's m. k_numbers_of(i,
    // st): step st of the tile's tokens 16 i to 16 i + 15; ks: K's scales by
    // token, of each step or one.
    // HOLD: the numbers are made there and then, and the compiler is not to make
    // those of all tokens before their products, for want of registers.
    template <bool HOLD, class F>
    __device__ __forceinline__ void scores(f32x4 (&x)[NT][4], const F& k_numbers_of, const float (*ks)[64], uint32_t kq)
    {
        scores<HOLD>(x, k_numbers_of, ks, kq, [&](int t, int st) { return start[t][st]; });
    }
    // start_of: where the start's numbers are kept
    template <bool HOLD, class F, class G>
    __device__ __forceinline__ void scores(f32x4 (&x)[NT][4], const F& k_numbers_of, const float (*ks)[64], uint32_t kq,
                                           const G& start_of)
    {
        if constexpr (KF) {
#pragma unroll
            for (int st = 0; st < KW; ++st) {
                f32x4 c[HK][NT];
#pragma unroll
                for (int half = 0; half < HK; ++half)
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        float one = start_of(t, st * HK + half);
                        if (HOLD) asm volatile("" : "+v"(one));    // made here, not kept as four
                        c[half][t] = f32x4{one, one, one, one};
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const v4u k = k_numbers_of(i, st);
#pragma unroll
                    for (int half = 0; half < HK; ++half) {
                        const f32x4 s = *reinterpret_cast<const f32x4*>(&ks[st * HK + half][16 * i + 4 * kq]);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const f32x4 d = attn_mfma<DT>(k, q[t][st * HK + half], c[half][t]);
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                x[t][i][r] = __builtin_fmaf(d[r], s[r], st == 0 && half == 0 ? -less[t] : x[t][i][r]);
                        }
                    }
                    if (HOLD && (i & 1)) __builtin_amdgcn_sched_barrier(0);
                }
            }
        } else {
            f32x4 scale[4], c[NT];
#pragma unroll
            for (int i = 0; i < 4; ++i) scale[i] = *reinterpret_cast<const f32x4*>(&ks[0][16 * i + 4 * kq]);
#pragma unroll
            for (int t = 0; t < NT; ++t) c[t] = f32x4{start_of(t, 0), start_of(t, 0), start_of(t, 0), start_of(t, 0)};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int st = 0; st < KW; ++st) {
                    const v4u k = k_numbers_of(i, st);
#pragma unroll
                    for (int t = 0; t < NT; ++t) x[t][i] = attn_mfma<DT>(k, q[t][st], st == 0 ? c[t] : x[t][i]);
                }
                if (HOLD) __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) x[t][i][r] = __builtin_fmaf(x[t][i][r], scale[i][r], -less[t]);
        }
    }

    // Tokens of the tile at `base` that are not there (valid: a bit each) or come
    // after a row's own.
    __device__ __forceinline__ void hide(f32x4 (&x)[NT][4], uint32_t base, uint64_t valid, uint32_t kq)
    {
        // most tiles have nothing to hide: this keeps the comparisons in the
        // caller's branch
        int32_t tile = __builtin_amdgcn_readfirstlane((int)base);
        asm volatile("" : "+s"(tile));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t bits = (uint32_t)(valid >> (16 * i + 4 * kq));
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int32_t tok = tile + (int32_t)(16 * i + 4 * kq + r);
#pragma unroll
                for (int t = 0; t < NT; ++t) x[t][i][r] = ((bits >> r) & 1u) && tok <= last[t] ? x[t][i][r] : kAttnNone;
            }
        }
    }

    // The weights exp(x - m), in x's place; keep: what the sums before are worth
    // now, where moved.
    __device__ __forceinline__ void weigh(f32x4 (&x)[NT][4], float (&keep)[NT], bool (&moved)[NT])
    {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float most = max3(x[t][0][0], x[t][0][1], x[t][0][2]);
#pragma unroll
            for (int k = 3; k < 15; k += 2) most = max3(most, x[t][k / 4][k % 4], x[t][(k + 1) / 4][(k + 1) % 4]);
            most = column_max(fmaxf(most, x[t][3][3]));
            keep[t] = 1.0f;
            moved[t] = __any(most > (m[t] == kAttnNone ? kAttnNone : 6.0f));
            if (moved[t]) {
                const float now = fmaxf(m[t], most + less[t]);
                keep[t] = now == m[t] ? 1.0f : exp2f(m[t] - now);
                m[t] = now;
                const float was = less[t];
                less[t] = now == kAttnNone ? 0.0f : now;
                const float more = less[t] - was;
                l[t] *= keep[t];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) x[t][i][r] -= more;
            }
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    x[t][i][r] = __builtin_amdgcn_exp2f(x[t][i][r]);
                    sum += x[t][i][r];
                }
            l[t] += sum;
        }
        __builtin_amdgcn_sched_barrier(0);
    }

    // Weights times scales, by the product whose 0 times anything is 0: a scale
    // that is no number reaches only the rows that see its token. (Its operands
    // come from LDS and from sums that have waited for the exponentials.)
    __device__ __forceinline__ static f32x4 scaled(const f32x4& x, const float* vs)
    {
        const f32x4 v = *reinterpret_cast<const f32x4*>(vs);
        return f32x4{mul_or_0(x[0], v[0]), mul_or_0(x[1], v[1]), mul_or_0(x[2], v[2]), mul_or_0(x[3], v[3])};
    }

    // By segments: the weights times V's scales, in fp16, and o^T += V^T P^T, 32
    // tokens a product. v_numbers_of(h, i): product i's V of half h of the tokens;
    // vs: V's scales by token, of each segment or one.
    template <bool HOLD, class F>
    __device__ __forceinline__ void add(const f32x4 (&x)[NT][4], const float (&keep)[NT], const bool (&moved)[NT], const F& v_numbers_of,
                                        const float (*vs)[64], uint32_t kq, uint32_t lane)
    {
        add<HOLD>(x, keep, moved, v_numbers_of, vs, kq, lane, [&](int t, int g) -> float& { return top[t][g]; });
    }
    // top_of: where the largest weights are kept
    template <bool HOLD, class F, class G>
    __device__ __forceinline__ void add(const f32x4 (&x)[NT][4], const float (&keep)[NT], const bool (&moved)[NT], const F& v_numbers_of,
                                        const float (*vs)[64], uint32_t kq, uint32_t lane, const G& top_of)
    {
        constexpr int T = VT / NGV * HV;           // products of a segment
        const uint32_t low = (lane & 8) ? 0u : ~0u;        // rows of its first half
#pragma unroll
        for (int seg = 0; seg < NGV / HV; ++seg) {
            v4u p[HV][NT][2];
#pragma unroll
            for (int half = 0; half < HV; ++half) {
                const int g = seg * HV + half;
                // Weights are at most 2^6 (m follows beyond that): the tile's scales
                // tell whether one could outgrow fp16. If so, or where a maximum has
                // moved, the powers of two are set anew from the largest product.
                bool set = __any(fabsf(vs[g][lane]) > safe[g]);
#pragma unroll
                for (int t = 0; t < NT; ++t) set = set || moved[t];
                if (set) {
                    int32_t least = 127;
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        float high = 0.0f;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const f32x4 w = scaled(x[t][i], &vs[g][16 * i + 4 * kq]);
                            high = max3_abs(max3_abs(high, w[0], w[1]), w[2], w[3]);
                        }
                        high = fmaxf(top_of(t, g) * keep[t], column_max(high));
                        top_of(t, g) = high;
                        int32_t now = __builtin_amdgcn_frexp_expf(high);
                        now = high > 0.0f ? min(max(now, -120), 120) : e[t][g];
                        float f = __builtin_ldexpf(keep[t], e[t][g] - now);
                        e[t][g] = now;
                        least = min(least, now);
                        if (HV == 2) f = (half == 0) == (kq < 2) ? f : 1.0f;
#pragma unroll
                        for (int i = 0; i < T; ++i) acc[t][seg * T + i] *= f;
                    }
                    safe[g] = __builtin_ldexpf(0x1p9f, least16(least));    // 2^6 * 2^9 = 2^15
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    f32x4 w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = scaled(x[t][i], &vs[g][16 * i + 4 * kq]);
                    const float c = __builtin_ldexpf(1.0f, -e[t][g]);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const f32x4& v = w[2 * h + (j >> 1)];
                            const f32x2 pair{v[2 * (j & 1)] * c, v[2 * (j & 1) + 1] * c};
                            p[half][t][h][j] = Store<ROPE_DTYPE_F16>::narrow(pair);
                        }
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = seg * T; i < (seg + 1) * T; ++i) {
                    const v4u v = v_numbers_of(h, i);
#pragma unroll
                    for (int half = 0; half < HV; ++half) {
                        const uint32_t rows = half == 0 ? low : ~low;
                        const v4u of = HV == 1 ? v : v4u{v[0] & rows, v[1] & rows, v[2] & rows, v[3] & rows};
#pragma unroll
                        for (int t = 0; t < NT; ++t) acc[t][i] = attn_mfma<ROPE_DTYPE_F16>(of, p[half][t][h], acc[t][i]);
                    }
                    if (HOLD && (i & 1)) __builtin_amdgcn_sched_barrier(0);
                }
        }
    }

    // The power of two of product i's sums.
    __device__ __forceinline__ int32_t power(int t, int i, uint32_t kq) const
    {
        if constexpr (HV == 2) return kq < 2 ? e[t][i & ~1] : e[t][i | 1];
        else return e[t][VF ? i / 2 : 0];
    }

    // Lane j of v that product i's row 4 kq + r holds.
    __device__ __forceinline__ static uint32_t lane_of(int i, int r, uint32_t kq)
    {
        return VF ? 32 * (i >> 1) + 8 * kq + 2 * r + (i & 1) : VT * (4 * kq + r) + i;
    }

    // The rows' results, or (split) their part of them.
    __device__ __forceinline__ void store(const AttnArgs& a, const AttnAt& at, uint32_t head, uint32_t r0, uint32_t live, uint32_t n16,
                                          uint32_t kq)
    {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint32_t r = r0 + t * 16 + n16;
            const float sum = column_sum(l[t]);
            if (r >= live) continue;
            const uint32_t s = fast_div(r, a.rep_div), h = head * a.rep + (r - s * a.rep);
            const float inv = a.split ? 1.0f : one_over(sum);
            const uint64_t row = part_row(a, at.part, s, h);
            gchar* dst = as_global(a.out.data) + (at.b * a.out.sb + s * a.out.ss + h * a.out.sn) * 2;
#pragma unroll
            for (int c = 0; c < VT / 2; ++c) {     // 8 consecutive lanes
                const float f = __builtin_ldexpf(inv, power(t, 2 * c, kq));
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] = f * (VF ? acc[t][2 * c + (k & 1)][k >> 1] : acc[t][(8 * c + k) % VT][(8 * c + k) / VT]);
                const uint32_t j = VF ? 32 * c + 8 * kq : 4 * VT * kq + 8 * c;
                if (j >= a.Dv) continue;
                if (!a.split) store_chunk<DT>(dst + j * 2, v);
                else store_chunk<ROPE_DTYPE_F32>(as_global(a.part + row * a.Dv + j), v);
            }
            if (a.split && kq == 0) part_stats(a)[row] = make_float2(m[t], sum);
        }
    }
};

// Where a tile's tokens are: a lane a token.
struct AttnPlace {
    uint32_t page, in_page;                        // page 0 where there is none
    bool there;
};

__device__ __forceinline__ AttnPlace attn_look_up(const AttnArgs& a, const int32_t* table, uint32_t tok, uint32_t to)
{
    AttnPlace p{0, 0, false};
    if (tok < to) {
        const uint32_t col = fast_div(tok, a.page_div);
        p.page = (uint32_t)table[col];
        p.in_page = tok - col * a.page_div.d;
        p.there = true;
    }
    return p;
}

// (apart from the look-up, so as not to wait for it there)
__device__ __forceinline__ void attn_settle(const AttnArgs& a, AttnPlace& p)
{
    p.there = p.there && p.page < a.page_limit;
    p.page = p.there ? p.page : 0;
    p.in_page = p.there ? p.in_page : 0;
}

// The first row of 16 tokens that stand in one page, as a scalar address.
__device__ __forceinline__ const gchar* attn_group_at(const AttnPlace& p, int i, const gchar* base, const CacheRef& c)
{
    const uint32_t page = __builtin_amdgcn_readlane((int)p.page, 16 * i);
    const uint32_t in_page = __builtin_amdgcn_readlane((int)p.in_page, 16 * i);
    return base + (int64_t)page * c.st[0] + (int64_t)in_page * c.st[1];
}

// An offset that the compiler cannot widen outside of a loop: a load then takes
// it as it is, beside its scalar address.
__device__ __forceinline__ uint32_t attn_offset(uint32_t v)
{
    asm volatile("" : "+v"(v));
    return v;
}

// This lane's number, made anew: a register less over a loop.
__device__ __forceinline__ uint32_t attn_lane()
{
    uint32_t v;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(v));
    return v;
}

// Where a register of a lane's V starts in its row: 4 bytes (2 of rows of up to
// 64 lanes) that end with the row, or the first ones.
template <int DVP, int VF>
__device__ __forceinline__ uint32_t attn_v_byte(uint32_t n16, int c, uint32_t v_bytes)
{
    const uint32_t off = VF ? (DVP == 64 ? 16 * (n16 & 1) + 2 * (n16 >> 1) : 64 * c + 16 * (n16 & 3) + 4 * (n16 >> 2))
                            : DVP == 64 ? 2 * n16 : DVP / 32 * n16 + 4 * c;
    return off < v_bytes ? off : 0;
}

// The tokens that the rows r0 to r1 - 1 see, and those that all of them see.
struct AttnSpan {
    uint32_t some, all;
};
__device__ __forceinline__ AttnSpan attn_span(const AttnArgs& a, const AttnSeq& seq, uint32_t r0, uint32_t r1)
{
    AttnSpan s{(uint32_t)seq.tokens, (uint32_t)seq.tokens};
    if (a.causal) {
        s.some = (uint32_t)max((int64_t)0, min((int64_t)s.some, seq.first + fast_div(r1 - 1, a.rep_div) + 1));
        s.all = (uint32_t)max((int64_t)0, min((int64_t)s.all, seq.first + fast_div(r0, a.rep_div) + 1));
    }
    return s;
}

// Waves that a SIMD is to hold: what their registers allow.
constexpr int attn_waves(int lanes, int kf, int tiles)
{
    return lanes == 256 || kf == kHalves ? 1 : lanes == 64 ? 4 - tiles : kf && tiles == 2 ? 1 : 2;
}

template <int DT, int DP, int DVP, int KF, int VF, bool P16, int NT>
__global__ void __launch_bounds__(256, attn_waves(DVP, KF, NT)) rope_attn_mfma_kernel(AttnVecArgs a)
{
    using Lds = AttnLds<DP, DVP, KF, VF, NT>;
    using R = AttnRows<DT, DP, DVP, KF, VF, NT>;
    constexpr int KW = R::KW;                      // words of a K row that a lane takes
    constexpr int VT = R::VT;
    constexpr int VR = DVP >= 128 ? DVP / 128 : 1; // registers of a token's V
    constexpr int VH = DVP / 64;                   // 16-bit halves of them
    constexpr int NGK = Lds::NGK, NGV = Lds::NGV;
    __shared__ Lds lds;
    const uint32_t lane = threadIdx.x & 63, n16 = lane & 15, kq = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    typename Lds::Wave& my = lds.wave[wave];

    AttnAt at;
    if (!attn_at(a, blockIdx.x, &at)) return;      // the same for the whole block
    const AttnSeq seq = attn_seq(a, at.b);
    const uint32_t head_wave = wave & (a.head_waves - 1), token_wave = a.row_waves > 1 ? 0 : wave / a.head_waves;
    const uint32_t head = at.head * a.head_waves + head_wave, waves = a.token_waves;
    const uint32_t r0 = (at.tile * a.row_waves + (a.row_waves > 1 ? wave : 0)) * 16 * NT;
    const uint32_t live = min(a.rows, (uint32_t)seq.count * a.rep);
    if (r0 >= live) return;                        // where waves are joined the same for the whole block
    const AttnSpan span = attn_span(a, seq, r0, min(r0 + 16 * NT, live));
    uint32_t from, to;
    attn_part(at, span.some, &from, &to);
    const uint32_t all = min(span.all, to);
    R rows;
    rows.load(a, seq, at.b, head, r0, live, n16, kq);

    // where this lane's words of a row start
    const gchar* const k_base = as_global(a.kc.data) + head * a.kc.st[2];
    const gchar* const v_base = as_global(a.vc.data) + head * a.vc.st[2];
    const gchar* const ks_base = as_global(a.kc.scales) + head * a.kc.sc[2] * 4;
    const gchar* const vs_base = as_global(a.vc.scales) + head * a.vc.sc[2] * 4;
    const int32_t* const table = a.table + at.b * a.table_stride;
    const uint32_t k_bytes = a.D / 2, v_bytes = a.Dv / 2;
    const uint32_t sel1 = (lane & 1) ? 0x03070105u : 0x06020400u;
    const uint32_t sel2 = (lane & 2) ? 0x03020706u : 0x05040100u;

    uint32_t kw[4][KW], vw[16][VR];
    float ks[NGK], vs[NGV];
    bool there = false;
    // Where 16 consecutive tokens stand in one page (P16) their rows start at one
    // scalar address, and a lane's words at offsets from it that do not change;
    // else each row's address comes from the lane that has its token.
    const uint32_t k_step = n16 * (uint32_t)a.kc.st[1], v_step = 4 * kq * (uint32_t)a.vc.st[1];
    // the scales and K's codes of a tile whose pages are known
    const auto fetch_k = [&](AttnPlace& p) {
        attn_settle(a, p);
        there = p.there;
        const int64_t page = p.page, in_page = p.in_page;
        const gchar* sk = ks_base + (page * a.kc.sc[0] + in_page * a.kc.sc[1]) * 4;
        const gchar* sv = vs_base + (page * a.vc.sc[0] + in_page * a.vc.sc[1]) * 4;
#pragma unroll
        for (int g = 0; g < NGK; ++g) {
            const uint32_t at_g = KF ? min((uint32_t)(g * attn_group(KF)) / a.k_group, a.k_groups - 1) : 0;
            ks[g] = there ? gload<float>(sk + at_g * 4) : 0.0f;
        }
#pragma unroll
        for (int g = 0; g < NGV; ++g) {
            const uint32_t at_g = VF ? min((uint32_t)(g * attn_group(VF)) / a.v_group, a.v_groups - 1) : 0;
            vs[g] = there ? gload<float>(sv + at_g * 4) : 0.0f;
        }
        if constexpr (!P16) {
            my.k_at[lane] = page * a.kc.st[0] + in_page * a.kc.st[1];
            my.v_at[lane] = page * a.vc.st[0] + in_page * a.vc.st[1];
            wave_sync();
        }
        uint32_t k_off[KF ? KW : 1];
#pragma unroll
        for (int st = 0; st < (KF ? KW : 1); ++st) {
            const uint32_t off = KF ? 16 * st + 4 * kq : 4 * KW * kq;
            k_off[st] = attn_offset((P16 ? k_step : 0) + (off < k_bytes ? off : 0));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const gchar* row = P16 ? attn_group_at(p, i, k_base, a.kc) : k_base + my.k_at[16 * i + n16];
            if constexpr (KF) {
#pragma unroll
                for (int st = 0; st < KW; ++st) kw[i][st] = gload<uint32_t>(row + k_off[st]);
            } else if constexpr (KW == 2) {
                const v2u w = gload<v2u>(row + k_off[0]);
                kw[i][0] = w[0];
                kw[i][1] = w[1];
            } else {
#pragma unroll
                for (int c = 0; c < KW / 4; ++c) {
                    const v4u w = gload<v4u>(row + k_off[0] + 16 * c);
#pragma unroll
                    for (int j = 0; j < 4; ++j) kw[i][4 * c + j] = w[j];
                }
            }
        }
    };
    const auto fetch_v = [&](const AttnPlace& p) {
        const gchar* group[4];
        if constexpr (P16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) group[i] = attn_group_at(p, i, v_base, a.vc);
        }
        uint32_t v_off[P16 ? 4 : 1][VR];
#pragma unroll
        for (int c = 0; c < VR; ++c)
#pragma unroll
            for (int r = 0; r < (P16 ? 4 : 1); ++r)
                v_off[r][c] = attn_offset((P16 ? v_step + r * (uint32_t)a.vc.st[1] : 0) + attn_v_byte<DVP, VF>(n16, c, v_bytes));
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const gchar* row = P16 ? group[i >> 2] : v_base + my.v_at[16 * (i >> 2) + 4 * kq + (i & 3)];
#pragma unroll
            for (int c = 0; c < VR; ++c) {
                const gchar* at = row + v_off[P16 ? i & 3 : 0][c];
                if constexpr (DVP == 64) vw[i][c] = gload<uint16_t>(at);
                else vw[i][c] = gload<uint32_t>(at);
            }
        }
    };

    const Numbers k_const = k_constants<DT>();
    const VConstants v_const = v_constants();
    const uint32_t step = 64 * waves;
    uint32_t base = from + 64 * token_wave;
    AttnPlace next = attn_look_up(a, table, base + lane, to);
    if (base < to) {
        fetch_k(next);
        fetch_v(next);
    }
    next = attn_look_up(a, table, (base + step < base ? to : base + step) + lane, to);
    for (; base < to; base += step) {
        // the tile's scales, by token, and its codes
        const uint64_t valid = __ballot(there);
#pragma unroll
        for (int g = 0; g < NGK; ++g) my.ks[g][lane] = ks[g] * a.scale2;
#pragma unroll
        for (int g = 0; g < NGV; ++g) my.vs[g][lane] = vs[g];
        wave_sync();

        f32x4 x[NT][4];
        rows.template scores<true>(x, [&](int i, int st) { return k_numbers<DT>(kw[i][st], k_const); }, my.ks, kq);
        if (base + 64 > all || valid != ~0ull) rows.hide(x, base, valid, kq);

        // The next tile's scales and K; its V when this one's is used up. (Behind
        // the last tile nothing new: a branch around the loads would cost a copy
        // of their registers in every tile.)
        fetch_k(next);
        const AttnPlace after = attn_look_up(a, table, (to - base > 2 * step ? base + 2 * step : to) + lane, to);
        __builtin_amdgcn_sched_barrier(0);

        float keep[NT];
        bool moved[NT];
        rows.weigh(x, keep, moved);

        // V's words, the codes of two tokens at equal nibbles of their halves
        uint32_t two[2][VH][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = 8 * h + 4 * (j >> 1) + 2 * (j & 1);
                if constexpr (DVP == 64) {
                    uint32_t w = vw[i][0] | (vw[i + 1][0] << 16);
                    if constexpr (VF) {            // two lanes exchange bytes of both halves
                        const uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)w, 0xB1, 0xF, 0xF, true);
                        w = __builtin_amdgcn_perm(o, w, sel1);
                    }
                    two[h][0][j] = w;
                } else {
#pragma unroll
                    for (int c = 0; c < VR; ++c) {
                        uint32_t w0 = vw[i][c], w1 = vw[i + 1][c];
                        if constexpr (VF) {
                            w0 = quad_bytes(w0, sel1, sel2);
                            w1 = quad_bytes(w1, sel1, sel2);
                        }
                        two[h][2 * c][j] = __builtin_amdgcn_perm(w1, w0, 0x05040100);
                        two[h][2 * c + 1][j] = __builtin_amdgcn_perm(w1, w0, 0x07060302);
                    }
                }
            }

        rows.template add<true>(x, keep, moved, [&](int h, int i) {
            v4u v;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t w = two[h][i >> 2][j];
                v[j] = (i & 3) == 0 ? v_numbers<0>(w, v_const) : (i & 3) == 1 ? v_numbers<1>(w, v_const) :
                       (i & 3) == 2 ? v_numbers<2>(w, v_const) : v_numbers<3>(w, v_const);
            }
            return v;
        }, my.vs, kq, lane);
        fetch_v(next);
        next = after;
    }

    if (waves == 1) {
        rows.store(a, at, head, r0, live, n16, kq);
        return;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const float sum = column_sum(rows.l[t]);
        __syncthreads();                           // the tiles (or the rows before) are done with this memory
        if (kq == 0) {
            lds.join.m[wave][n16] = rows.m[t];
            lds.join.l[wave][n16] = sum;
        }
        __syncthreads();
        float most = kAttnNone;
        for (uint32_t w = head_wave; w < 4; w += a.head_waves) most = fmaxf(most, lds.join.m[w][n16]);
        const float keep = part_weight(rows.m[t], most);
#pragma unroll
        for (int i = 0; i < VT; ++i) {
            const float f = __builtin_ldexpf(keep, rows.power(t, i, kq));
#pragma unroll
            for (int r = 0; r < 4; ++r) lds.join.o[wave][n16][R::lane_of(i, r, kq)] = rows.acc[t][i][r] * f;
        }
        __syncthreads();
        // 16 threads a row, 8 lanes at a time
        const uint32_t row16 = threadIdx.x >> 4, r = r0 + t * 16 + row16;
        const uint32_t s = fast_div(min(r, live - 1), a.rep_div);
        for (uint32_t hw = 0; hw < a.head_waves; ++hw) {
            float high = kAttnNone, whole = 0.0f;
            for (uint32_t w = hw; w < 4; w += a.head_waves) high = fmaxf(high, lds.join.m[w][row16]);
            for (uint32_t w = hw; w < 4; w += a.head_waves) {
                const float mw = lds.join.m[w][row16];
                whole += lds.join.l[w][row16] * part_weight(mw, high);
            }
            const uint32_t h = (at.head * a.head_waves + hw) * a.rep + (r - s * a.rep);
            const float inv = a.split ? 1.0f : one_over(whole);
            const uint64_t row = part_row(a, at.part, s, h);
            gchar* dst = as_global(a.out.data) + (at.b * a.out.sb + s * a.out.ss + h * a.out.sn) * 2;
            for (uint32_t j = 8 * (threadIdx.x & 15); j < a.Dv && r < live; j += 128) {
                float v[8] = {};
                for (uint32_t w = hw; w < 4; w += a.head_waves)
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] += lds.join.o[w][row16][j + k];
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] *= inv;
                if (!a.split) store_chunk<DT>(dst + j * 2, v);
                else store_chunk<ROPE_DTYPE_F32>(as_global(a.part + row * a.Dv + j), v);
            }
            if (a.split && r < live && (threadIdx.x & 15) == 0) part_stats(a)[row] = make_float2(high, whole);
        }
    }
}


// ---------------------------------------------------------------------------
// Many rows (a prompt's): the four waves of a block have 32 rows each (NT 2; 16
// where scales of 16 lanes leave no registers for more) of one cached head and go through the same tiles, so each makes numbers of a quarter
// of a tile, for all, in LDS: in the order in which the products take them, 16
// bytes a lane, so that no read or write meets another's bank. Numbers cost a
// wave 75 operations a tile then, not 300, of 700. Two buffers: while a tile is
// used the next one's numbers are made, its words having been loaded the tile
// before; one barrier a tile. 3 sequences of 2039 new tokens behind up to 4096
// others, 32 heads on 8 of 128 lanes: 480 us, 606 by waves on their own; with a
// scale for 32 lanes 858, 1106. (32 rows a wave: 48 and 64 were slower, for want
// of registers.)
// ---------------------------------------------------------------------------
template <int DP, int KF, int VF, bool P16, int NT>
struct alignas(16) AttnSharedLds {
    static constexpr int NGK = attn_groups(KF, DP), NGV = attn_groups(VF, DP);
    struct Buffer {
        v4u k[4][DP / 32][64];
        v4u v[2][DP / 16][64];
        float ks[NGK][64], vs[NGV][64];
    };
    Buffer tile[2];
    struct Where {
        int64_t k_at[64], v_at[64];
    };
    Where where[P16 ? 1 : 4];
    struct Wave {
        float start[NT][NGK][16], top[NT][NGV][16];    // the rows', where registers are short
    };
    Wave wave[4];
};

template <int DT, int DP, int KF, int VF, bool P16, int NT>
__global__ void __launch_bounds__(256, 2) rope_attn_shared_kernel(AttnVecArgs a)
{
    using Lds = AttnSharedLds<DP, KF, VF, P16, NT>;
    using R = AttnRows<DT, DP, DP, KF, VF, NT>;
    constexpr int KW = R::KW, VT = R::VT, NGK = Lds::NGK, NGV = Lds::NGV;
    static_assert(DP == 64 || DP == 128, "a register a token's V");
    __shared__ Lds lds;
    const uint32_t lane = threadIdx.x & 63, n16 = lane & 15, kq = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    AttnAt at;
    if (!attn_at(a, blockIdx.x, &at)) return;      // the same for the whole block
    at.tile = a.tiles - 1 - at.tile;               // those that see the most tokens first
    const AttnSeq seq = attn_seq(a, at.b);
    const uint32_t block_row = at.tile * (64 * NT), r0 = block_row + wave * (16 * NT);
    const uint32_t live = min(a.rows, (uint32_t)seq.count * a.rep);
    if (block_row >= live) return;                 // the same for the whole block
    uint32_t from, to;
    attn_part(at, attn_span(a, seq, block_row, min(block_row + 64 * NT, live)).some, &from, &to);
    // (a wave without rows makes numbers only)
    const AttnSpan span = r0 < live ? attn_span(a, seq, r0, min(r0 + 16 * NT, live)) : AttnSpan{0, 0};
    const uint32_t all = min(span.all, to), some = min(span.some, to);
    R rows;
    rows.load(a, seq, at.b, at.head, min(r0, live - 1), live, n16, kq);
    typename Lds::Wave& my = lds.wave[wave];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int g = 0; g < NGK; ++g) my.start[t][g][n16] = rows.start[t][g];
#pragma unroll
        for (int g = 0; g < NGV; ++g) my.top[t][g][n16] = 0.0f;
    }

    const gchar* const k_base = as_global(a.kc.data) + at.head * a.kc.st[2];
    const gchar* const v_base = as_global(a.vc.data) + at.head * a.vc.st[2];
    const gchar* const ks_base = as_global(a.kc.scales) + at.head * a.kc.sc[2] * 4;
    const gchar* const vs_base = as_global(a.vc.scales) + at.head * a.vc.sc[2] * 4;
    const int32_t* const table = a.table + at.b * a.table_stride;
    const uint32_t k_bytes = a.D / 2, v_bytes = a.Dv / 2;
    const uint32_t sel1 = (lane & 1) ? 0x03070105u : 0x06020400u;
    const uint32_t sel2 = (lane & 2) ? 0x03020706u : 0x05040100u;
    const uint32_t k_step = n16 * (uint32_t)a.kc.st[1], v_step = 4 * kq * (uint32_t)a.vc.st[1];
    // this wave's quarter: K of tokens 16 wave on; V of half `half` of the
    // tokens, products `part` * VT / 2 on; the scales of group `wave`, where there
    // are so many
    const uint32_t half = wave >> 1, part = wave & 1;
    const uint32_t v_sel = part ? 0x07060302u : 0x05040100u;
    const Numbers k_const = k_constants<DT>();
    const VConstants v_const = v_constants();

    uint32_t kw[KW], vw[8];
    constexpr int SK = (NGK + 3) / 4, SV = (NGV + 3) / 4;  // scales' groups of a wave: wave, wave + 4
    float ks[SK] = {}, vs[SV] = {};
    bool there = false;
    const auto fetch = [&](AttnPlace& p) {
        attn_settle(a, p);
        there = p.there;
        const int64_t page = p.page, in_page = p.in_page;
#pragma unroll
        for (int n = 0; n < SK; ++n) {
            if (wave + 4 * n >= NGK) continue;
            const uint32_t g = KF ? min((wave + 4 * n) * attn_group(KF) / a.k_group, a.k_groups - 1) : 0;
            ks[n] = there ? gload<float>(ks_base + (page * a.kc.sc[0] + in_page * a.kc.sc[1] + g) * 4) : 0.0f;
        }
#pragma unroll
        for (int n = 0; n < SV; ++n) {
            if (wave + 4 * n >= NGV) continue;
            const uint32_t g = VF ? min((wave + 4 * n) * attn_group(VF) / a.v_group, a.v_groups - 1) : 0;
            vs[n] = there ? gload<float>(vs_base + (page * a.vc.sc[0] + in_page * a.vc.sc[1] + g) * 4) : 0.0f;
        }
        if constexpr (!P16) {
            lds.where[wave].k_at[lane] = page * a.kc.st[0] + in_page * a.kc.st[1];
            lds.where[wave].v_at[lane] = page * a.vc.st[0] + in_page * a.vc.st[1];
            wave_sync();
        }
        const gchar* row = P16 ? attn_group_at(p, wave, k_base, a.kc) : k_base + lds.where[wave].k_at[16 * wave + n16];
        if constexpr (KF) {
#pragma unroll
            for (int st = 0; st < KW; ++st) {
                const uint32_t off = 16 * st + 4 * kq;
                kw[st] = gload<uint32_t>(row + attn_offset((P16 ? k_step : 0) + (off < k_bytes ? off : 0)));
            }
        } else if constexpr (KW == 2) {
            const v2u w = gload<v2u>(row + attn_offset((P16 ? k_step : 0) + 8 * kq));
            kw[0] = w[0];
            kw[1] = w[1];
        } else {
            const v4u w = gload<v4u>(row + attn_offset((P16 ? k_step : 0) + 16 * kq));
#pragma unroll
            for (int j = 0; j < 4; ++j) kw[j] = w[j];
        }
        const uint32_t byte = attn_v_byte<DP, VF>(n16, 0, v_bytes);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const gchar* r = P16 ? attn_group_at(p, 2 * half + (i >> 2), v_base, a.vc)
                                 : v_base + lds.where[wave].v_at[32 * half + 16 * (i >> 2) + 4 * kq + (i & 3)];
            const uint32_t off = attn_offset((P16 ? v_step + (i & 3) * (uint32_t)a.vc.st[1] : 0) + byte);
            if constexpr (DP == 64) vw[i] = gload<uint16_t>(r + off);
            else vw[i] = gload<uint32_t>(r + off);
        }
    };
    // the words' numbers, and the scales, to a buffer
    const auto put = [&](typename Lds::Buffer& to_tile) {
#pragma unroll
        for (int st = 0; st < KW; ++st) to_tile.k[wave][st][lane] = k_numbers<DT>(kw[st], k_const);
        uint32_t two[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t w0 = vw[4 * (j >> 1) + 2 * (j & 1)], w1 = vw[4 * (j >> 1) + 2 * (j & 1) + 1];
            if constexpr (DP == 64) {
                uint32_t w = w0 | (w1 << 16);
                if constexpr (VF) {
                    const uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)w, 0xB1, 0xF, 0xF, true);
                    w = __builtin_amdgcn_perm(o, w, sel1);
                }
                two[j] = w >> (8 * part);
            } else {
                if constexpr (VF) {
                    w0 = quad_bytes(w0, sel1, sel2);
                    w1 = quad_bytes(w1, sel1, sel2);
                }
                two[j] = __builtin_amdgcn_perm(w1, w0, v_sel);
            }
        }
#pragma unroll
        for (int i = 0; i < VT / 2; ++i) {
            v4u v;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = i == 0 ? v_numbers<0>(two[j], v_const) : i == 1 ? v_numbers<1>(two[j], v_const) :
                       i == 2 ? v_numbers<2>(two[j], v_const) : v_numbers<3>(two[j], v_const);
            to_tile.v[half][part * (VT / 2) + i][lane] = v;
        }
#pragma unroll
        for (int n = 0; n < SK; ++n)
            if (wave + 4 * n < NGK) to_tile.ks[wave + 4 * n][lane] = ks[n] * a.scale2;
#pragma unroll
        for (int n = 0; n < SV; ++n)
            if (wave + 4 * n < NGV) to_tile.vs[wave + 4 * n][lane] = vs[n];
    };

    AttnPlace next = attn_look_up(a, table, from + lane, to);
    uint64_t valid = 0;
    if (from < to) {
        fetch(next);
        valid = __ballot(there);
        put(lds.tile[0]);
        next = attn_look_up(a, table, from + 64 + lane, to);
        fetch(next);
        next = attn_look_up(a, table, (to - from > 128 ? from + 128 : to) + lane, to);
    }
    __syncthreads();
    uint32_t buffer = 0;
    for (uint32_t base = from; base < to; base += 64) {
        const typename Lds::Buffer& tile = lds.tile[buffer];
        const uint64_t next_valid = __ballot(there);
        f32x4 x[NT][4];
        float keep[NT];
        bool moved[NT];
        const bool used = base < some;
        if (used) {
            rows.template scores<false>(x, [&](int i, int st) { return tile.k[i][st][lane]; }, tile.ks, kq,
                                        [&](int t, int st) { return my.start[t][st][n16]; });
            if (base + 64 > all || valid != ~0ull) rows.hide(x, base, valid, kq);
            rows.weigh(x, keep, moved);
        }
        // (behind the last tile nothing new is made or loaded, but it costs no
        // branch)
        put(lds.tile[buffer ^ 1]);
        fetch(next);
        next = attn_look_up(a, table, (to - base > 192 ? base + 192 : to) + lane, to);
        __builtin_amdgcn_sched_barrier(0);
        if (used) rows.template add<false>(x, keep, moved, [&](int h, int i) { return tile.v[h][i][lane]; }, tile.vs, kq, lane,
                                     [&](int t, int g) -> float& { return my.top[t][g][n16]; });
        valid = next_valid;
        buffer ^= 1;
        __syncthreads();
    }
    if (r0 < live) rows.store(a, at, at.head, r0, live, n16, kq);
}

// ---------------------------------------------------------------------------
// Few rows, four cached heads beside each other: a block's waves have a head
// each, and load a tile's rows for all four, straight to LDS, while the tile
// before is used: 256 (128) consecutive bytes a token and 16 of scales, where
// each wave for itself would ask for 64 (32) and 4. The card brings the first
// at the rate of a copy, not the second. 64 sequences of 1 to 8192 tokens, 32
// heads on 8 of 128: 105 us (4.1 TB/s), 119 by waves on their own, whose loads
// alone, without arithmetic, are 115; 64 heads on 16 of 64: 132 us, 203. A
// token's 16-byte pieces stand in LDS in an order that its number turns, so
// that neither K's reads (the same piece of 16 tokens) nor V's (four pieces of
// four tokens) meet in a bank. Two buffers of 17 or 35 KB; one barrier a tile.
// ---------------------------------------------------------------------------
template <int DP, int KF, int VF, int NT>
struct alignas(16) AttnHeadsLds {
    static constexpr int kRow = 2 * DP;            // bytes of a token's four rows
    static constexpr bool kScales = !KF && !VF;    // one a row: they come with the codes
    static constexpr bool kRows = KF != kHalves || VF != kHalves;
    static constexpr int NGK = attn_groups(KF, DP), NGV = attn_groups(VF, DP);
    struct Tile {
        char k[64 * kRow], v[64 * kRow];
        float ks[kScales ? 64 : 0][4], vs[kScales ? 64 : 0][4];
    };
    Tile tile[2];
    struct Wave {
        float ks[NGK][64], vs[NGV][64];
        // the rows', where registers are short (where scales leave room for them)
        float start[kRows ? NT : 0][NGK][16], top[kRows ? NT : 0][NGV][16];
    };
    Wave wave[4];
};

template <int DT, int DP, int KF, int VF, int NT>
__global__ void __launch_bounds__(256, 2) rope_attn_heads_kernel(AttnVecArgs a)
{
    using Lds = AttnHeadsLds<DP, KF, VF, NT>;
    using R = AttnRows<DT, DP, DP, KF, VF, NT>;
    constexpr int KW = R::KW, NGK = Lds::NGK, NGV = Lds::NGV;
    constexpr uint32_t kPieces = Lds::kRow / 16;   // of a token
    constexpr uint32_t kTokens = 64 / kPieces;     // of a load
    constexpr int kLoads = 16 / kTokens;           // of 16 tokens
    static_assert(DP == 64 || DP == 128, "whole loads of 16 tokens");
    __shared__ Lds lds;
    const uint32_t lane = threadIdx.x & 63, n16 = lane & 15, kq = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    AttnAt at;
    if (!attn_at(a, blockIdx.x, &at)) return;      // the same for the whole block
    const AttnSeq seq = attn_seq(a, at.b);
    const uint32_t head0 = at.head * 4, head = head0 + wave, r0 = at.tile * 16 * NT;
    const uint32_t live = min(a.rows, (uint32_t)seq.count * a.rep);
    if (r0 >= live) return;                        // the same for the whole block
    const AttnSpan span = attn_span(a, seq, r0, min(r0 + 16 * NT, live));
    uint32_t from, to;
    attn_part(at, span.some, &from, &to);
    const uint32_t all = min(span.all, to);
    R rows;
    rows.load(a, seq, at.b, head, r0, live, n16, kq);

    const gchar* const k_base = as_global(a.kc.data) + head0 * a.kc.st[2];
    const gchar* const v_base = as_global(a.vc.data) + head0 * a.vc.st[2];
    const gchar* const ks_base = as_global(a.kc.scales) + (Lds::kScales ? head0 : head) * a.kc.sc[2] * 4;
    const gchar* const vs_base = as_global(a.vc.scales) + (Lds::kScales ? head0 : head) * a.vc.sc[2] * 4;
    const int32_t* const table = a.table + at.b * a.table_stride;
    const uint32_t sel1 = (lane & 1) ? 0x03070105u : 0x06020400u;
    const uint32_t sel2 = (lane & 2) ? 0x03020706u : 0x05040100u;
    const uint32_t lds_base = (uint32_t)(uintptr_t)((__attribute__((address_space(3))) Lds*)&lds);
    // a load's lanes: token lane / pieces of its kTokens, piece lane % pieces in
    // its turned order
    const uint32_t tok0 = lane / kPieces, piece0 = 16 * ((lane % kPieces) ^ tok0);
    const uint32_t k_tok = tok0 * (uint32_t)a.kc.st[1], v_tok = tok0 * (uint32_t)a.vc.st[1];
    float ks[NGK], vs[NGV];
    // this wave's quarter of a tile: 16 tokens of K and V. Scales: of all rows by
    // the first two waves, or a lane's token's of this wave's head
    const auto issue = [&](const AttnPlace& p, uint32_t buffer) {
        const int64_t page = p.page, in_page = p.in_page;
        const gchar* sk = ks_base + (page * a.kc.sc[0] + in_page * a.kc.sc[1]) * 4;
        const gchar* sv = vs_base + (page * a.vc.sc[0] + in_page * a.vc.sc[1]) * 4;
        if constexpr (!Lds::kScales) {
#pragma unroll
            for (int g = 0; g < NGK; ++g) {
                const uint32_t at_g = KF ? min((uint32_t)(g * attn_group(KF)) / a.k_group, a.k_groups - 1) : 0;
                ks[g] = p.there ? gload<float>(sk + at_g * 4) : 0.0f;
            }
#pragma unroll
            for (int g = 0; g < NGV; ++g) {
                const uint32_t at_g = VF ? min((uint32_t)(g * attn_group(VF)) / a.v_group, a.v_groups - 1) : 0;
                vs[g] = p.there ? gload<float>(sv + at_g * 4) : 0.0f;
            }
        }
        const gchar* k_row = attn_group_at(p, wave, k_base, a.kc);
        const gchar* v_row = attn_group_at(p, wave, v_base, a.vc);
        const uint32_t to_tile = lds_base + (uint32_t)offsetof(Lds, tile) + buffer * (uint32_t)sizeof(typename Lds::Tile);
        const uint32_t mine = to_tile + wave * 16 * Lds::kRow;
        const auto load = [&](const gchar* row, int64_t step, uint32_t tok, uint32_t to_codes) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                lds_dma16((const void*)(row + (int64_t)(i * kTokens) * step),
                          (attn_offset(piece0) ^ (16 * ((i * kTokens) % kPieces))) + tok, to_codes + 1024 * i);
        };
        load(k_row, a.kc.st[1], k_tok, mine + (uint32_t)offsetof(typename Lds::Tile, k));
        load(v_row, a.vc.st[1], v_tok, mine + (uint32_t)offsetof(typename Lds::Tile, v));
        if constexpr (Lds::kScales) {
            if (wave == 0) lds_dma16_far((const void*)sk, to_tile + (uint32_t)offsetof(typename Lds::Tile, ks));
            if (wave == 1) lds_dma16_far((const void*)sv, to_tile + (uint32_t)offsetof(typename Lds::Tile, vs));
        }
    };

    const Numbers k_const = k_constants<DT>();
    const VConstants v_const = v_constants();
    typename Lds::Wave& my = lds.wave[wave];
    if constexpr (Lds::kRows) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int g = 0; g < NGK; ++g) my.start[t][g][n16] = rows.start[t][g];
#pragma unroll
            for (int g = 0; g < NGV; ++g) my.top[t][g][n16] = 0.0f;
        }
    }
    AttnPlace now = attn_look_up(a, table, from + lane, to);
    attn_settle(a, now);
    if (from < to) issue(now, 0);
    AttnPlace next = attn_look_up(a, table, (to - from > 64 ? from + 64 : to) + lane, to);
    uint32_t buffer = 0;
    for (uint32_t base = from; base < to; base += 64) {
        wait_vm<0>();                              // this wave's loads are there
        // ... and everyone's, and everyone is done with the other buffer. (A bare
        // barrier; the empty asm keeps this tile's reads behind it.)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        const uint64_t valid = __ballot(now.there);
        const typename Lds::Tile& tile = lds.tile[buffer];
        if constexpr (Lds::kScales) {
            my.ks[0][lane] = now.there ? tile.ks[lane][wave] * a.scale2 : 0.0f;
            my.vs[0][lane] = now.there ? tile.vs[lane][wave] : 0.0f;
        } else {
#pragma unroll
            for (int g = 0; g < NGK; ++g) my.ks[g][lane] = ks[g] * a.scale2;
#pragma unroll
            for (int g = 0; g < NGV; ++g) my.vs[g][lane] = vs[g];
        }
        attn_settle(a, next);
        if (to - base > 64) issue(next, buffer ^ 1);
        const AttnPlace after = attn_look_up(a, table, (to - base > 128 ? base + 128 : to) + attn_lane(), to);
        wave_sync();
        // (KF: a word a step, where it is used)
        const auto k_piece = [&](int i, uint32_t n) {
            return tile.k + (16 * i + n16) * Lds::kRow + 16 * ((wave * (DP / 32) + n) ^ (n16 % kPieces));
        };
        uint32_t kw[4][KF ? 1 : KW];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (KF) {
            } else if constexpr (KW == 4) {
                const v4u w = *reinterpret_cast<const v4u*>(k_piece(i, kq));
#pragma unroll
                for (int j = 0; j < 4; ++j) kw[i][j] = w[j];
            } else {
                const v2u w = *reinterpret_cast<const v2u*>(k_piece(i, kq >> 1) + 8 * (kq & 1));
                kw[i][0] = w[0];
                kw[i][1] = w[1];
            }
        }
        f32x4 x[NT][4];
        rows.template scores<true>(x, [&](int i, int st) {
            return k_numbers<DT>(KF ? *reinterpret_cast<const uint32_t*>(k_piece(i, st) + 4 * kq) : kw[i][KF ? 0 : st], k_const);
        }, my.ks, kq, [&](int t, int st) {
            if constexpr (Lds::kRows) return my.start[t][st][n16];
            else return rows.start[t][st];
        });
        if (base + 64 > all || valid != ~0ull) rows.hide(x, base, valid, kq);
        float keep[NT];
        bool moved[NT];
        rows.weigh(x, keep, moved);
        // V's words, the codes of two tokens at equal nibbles of their halves
        const uint32_t byte = attn_v_byte<DP, VF>(n16, 0, DP / 2);
        uint32_t two[2][DP / 64][4];
        const auto word = [&](uint32_t i) -> uint32_t {
            const uint32_t in16 = 4 * kq + (i & 3);
            const char* at_v = tile.v + (16 * (i >> 2) + in16) * Lds::kRow +
                               16 * ((wave * (DP / 32) + (byte >> 4)) ^ (in16 % kPieces)) + (byte & 15);
            if constexpr (DP == 64) return *reinterpret_cast<const uint16_t*>(at_v);
            else return *reinterpret_cast<const uint32_t*>(at_v);
        };
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t i = 8 * h + 4 * (j >> 1) + 2 * (j & 1);
                uint32_t w0 = word(i), w1 = word(i + 1);
                if constexpr (DP == 64) {
                    uint32_t w = w0 | (w1 << 16);
                    if constexpr (VF) {
                        const uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)w, 0xB1, 0xF, 0xF, true);
                        w = __builtin_amdgcn_perm(o, w, sel1);
                    }
                    two[h][0][j] = w;
                } else {
                    if constexpr (VF) {
                        w0 = quad_bytes(w0, sel1, sel2);
                        w1 = quad_bytes(w1, sel1, sel2);
                    }
                    two[h][0][j] = __builtin_amdgcn_perm(w1, w0, 0x05040100);
                    two[h][1][j] = __builtin_amdgcn_perm(w1, w0, 0x07060302);
                }
            }
        rows.template add<true>(x, keep, moved, [&](int h, int i) {
            v4u v;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t w = two[h][i >> 2][j];
                v[j] = (i & 3) == 0 ? v_numbers<0>(w, v_const) : (i & 3) == 1 ? v_numbers<1>(w, v_const) :
                       (i & 3) == 2 ? v_numbers<2>(w, v_const) : v_numbers<3>(w, v_const);
            }
            return v;
        }, my.vs, kq, lane, [&](int t, int g) -> float& {
            if constexpr (Lds::kRows) return my.top[t][g][n16];
            else return rows.top[t][g];
        });
        now = next;
        next = after;
        buffer ^= 1;
    }
    rows.store(a, at, head, r0, live, n16, kq);
}

}  // namespace
}  // namespace rope
