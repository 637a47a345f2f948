// rope_cache_kernels.hpp -- writing rotated keys and values to a paged,
// quantised cache, and reading them back.
// Included by rope_cache.hip, next to the host code that launches them.
//
// Mathematics. A group of G lanes z with largest finite magnitude m is held
// as codes and one fp32 scale s = m / Q, Q the format's largest value (448
// for e4m3, 127, 7): code = the value of the format nearest to z / s, ties to
// the even one. Halves of m and the like are common in 16-bit data, so exact
// ties are too, and a quotient rounded to fp32 before it is rounded to the
// code would send some of them the wrong way, or make a tie of a value next
// to one; quotient() keeps the side.
#pragma once

#include "rope_cache_plan.hpp"
#include "rope_pos_kernels.hpp"

namespace rope {
namespace {

constexpr int kFmtSame = 0;   // the rows' storage type
constexpr int kFmtE4M3 = ROPE_CACHE_E4M3;
constexpr int kFmtInt8 = ROPE_CACHE_INT8;
constexpr int kFmtInt4 = ROPE_CACHE_INT4;

template <int FMT> __device__ constexpr float fmt_max() { return FMT == kFmtE4M3 ? 448.0f : FMT == kFmtInt8 ? 127.0f : 7.0f; }

// Rows of q, k, v or out: row (b,s,n) at b*sb + s*ss + n*sn elements.
struct Rows {
    char* data;
    int64_t sb, ss, sn;
};

struct CacheRef {
    char* data;
    float* scales;
    int64_t st[3];    // bytes: page, slot, head
    int64_t sc[3];    // floats
    uint32_t group;   // lanes per scale
};

// cos and sin source of a call: positions on one or several axes.
struct Turn {
    const int64_t* pos;
    const double* inv_freq;
    int64_t sb, ss;
    PosAxes ax;
    int32_t tdt;            // type cos and sin are rounded to
    uint32_t start, L, half, pairs;
    FastDiv half_div;
};

// cos and sin of pair i of token (b, s), rounded to the table type.
__device__ __forceinline__ float2 turn_cos_sin(const Turn& t, uint32_t b, uint32_t s, uint32_t i)
{
    const int64_t p = axis_position(t.ax, t.pos + b * t.sb + s * t.ss, i);
    const double f = t.inv_freq[i];
    switch (t.tdt) {
    case ROPE_DTYPE_F32: return pos_cos_sin<ROPE_DTYPE_F32>(p, f);
    case ROPE_DTYPE_F16: return pos_cos_sin<ROPE_DTYPE_F16>(p, f);
    default: return pos_cos_sin<ROPE_DTYPE_BF16>(p, f);
    }
}

// The pair of slice lane j, and whether j is its first lane.
__device__ __forceinline__ uint32_t turn_pair(const Turn& t, uint32_t j, bool* first)
{
    const uint32_t h = fast_div(j, t.half_div);     // half-group number
    *first = (h & 1u) == 0;
    return (h >> 1) * t.half + (j - h * t.half);
}

// The scale of a group whose largest finite magnitude is m.
template <int FMT>
__device__ __forceinline__ float group_scale(float m)
{
    return m > 0.0f ? fmaxf(m / fmt_max<FMT>(), 0x1p-100f) : 1.0f;
}

// A float on the same side of every code and of every midpoint between two
// codes as the exact x / s, and equal to one only where x / s is. Codes and
// midpoints (t below) have at most 8 significant bits, so among fp32 numbers
// their significands are even. q is x / s within one unit in the last place
// (one Newton step on x * (1/s)) and e its residual, exact by the fused
// multiply-add. q odd: q is not a t and the nearest t are more than a unit
// away. q even and e not 0: one unit towards x / s makes it odd, and leaves
// it on the side where x / s lies. Quotients below 2^-12 round to zero in
// every format and are left alone, so the scale's floor of 2^-100 keeps
// every residual that decides out of the subnormals.
__device__ __forceinline__ float quotient(float x, float s, float inv)
{
    const float q0 = x * inv;
    const float q = __builtin_fmaf(__builtin_fmaf(-q0, s, x), inv, q0);
    const float e = __builtin_fmaf(-q, s, x);
    const uint32_t u = __float_as_uint(q);
    const uint32_t away = (__float_as_uint(e) ^ u) >> 31;          // 1: x / s lies nearer to zero
    const bool move = e != 0.0f && (u & 1u) == 0 && fabsf(q) >= 0x1p-12f;
    return __uint_as_float(move ? u + 1u - 2u * away : u);
}

// The code of lane value x (as a float that the format holds) in a group of
// largest finite magnitude m and scale s.
template <int FMT>
__device__ __forceinline__ float code_of(float x, float m, float s, float inv)
{
    const float c = fminf(fmaxf(x, -m), m);        // an infinity takes the code of +-m
    float q = quotient(c, s, inv);
    if constexpr (FMT != kFmtE4M3) q = rintf(q);
    q = fminf(fmaxf(q, -fmt_max<FMT>()), fmt_max<FMT>());
    if (x != x) q = FMT == kFmtE4M3 ? x : 0.0f;
    return q;
}

// The magnitude that x adds to its group's largest: 0 unless finite.
__device__ __forceinline__ float finite_mag(float x)
{
    const float a = fabsf(x);
    return a < __builtin_inff() ? a : 0.0f;
}

// Two codes as bytes (e4m3, int8; the low half of the result).
template <int FMT>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    if constexpr (FMT == kFmtE4M3) {
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false) & 0xFFFFu;
    } else {
        return ((uint32_t)(int)a & 0xFFu) | (((uint32_t)(int)b & 0xFFu) << 8);
    }
}

// ---------------------------------------------------------------------------
// General kernels: any dimensions, alignment, slice and group. One wave per
// row; the row's rotated values in LDS, its groups' largest magnitudes by LDS
// maxima (of the bits of non-negative floats: the order does not matter).
// ---------------------------------------------------------------------------
struct CacheWriteArgs {
    Rows q, k, v;
    CacheRef kc, vc;
    uint32_t Nq, Nk, Nv;      // rows of a token: q, then k, then v
    uint32_t Dk, Dv;
    uint32_t tokens, S;
    uint64_t rows;            // tokens * (Nq + Nk + Nv)
    const int64_t* slots;
    int64_t slot_sb, slot_ss;
    int64_t page_size, nslots;
    int32_t rotate_k;
    Turn turn;
    FastDiv s_div, row_div;   // by S and by the rows of a token
};

// A row's place: its token, kind (0 q, 1 k, 2 v) and head.
struct RowAt {
    uint32_t b, s, n;
    int kind;
};

__device__ __forceinline__ RowAt row_at(const CacheWriteArgs& a, uint32_t row)
{
    const uint32_t tok = fast_div(row, a.row_div);
    const uint32_t j = row - tok * a.row_div.d;
    RowAt r;
    r.b = fast_div(tok, a.s_div);
    r.s = tok - r.b * a.s_div.d;
    r.kind = j < a.Nq ? 0 : j < a.Nq + a.Nk ? 1 : 2;
    r.n = j - (r.kind == 0 ? 0 : r.kind == 1 ? a.Nq : a.Nq + a.Nk);
    return r;
}

constexpr int kGenThreads = 64;

template <int DT, int FMT>
__global__ void __launch_bounds__(kGenThreads) rope_cache_write_general_kernel(CacheWriteArgs a)
{
    __shared__ float z[ROPE_D_LIMIT];
    __shared__ uint32_t mag[ROPE_D_LIMIT / 2];
    const uint32_t t = threadIdx.x;
    for (uint64_t row64 = blockIdx.x; row64 < a.rows; row64 += gridDim.x) {
        const RowAt r = row_at(a, (uint32_t)row64);
        const Rows& src = r.kind == 0 ? a.q : r.kind == 1 ? a.k : a.v;
        const uint32_t D = r.kind == 2 ? a.Dv : a.Dk;
        int64_t slot = -1;
        if (r.kind != 0) {
            slot = a.slots[r.b * a.slot_sb + r.s * a.slot_ss];
            if (slot < 0 || slot >= a.nslots) continue;     // the same for the whole block
        }
        const int64_t off = r.b * src.sb + r.s * src.ss + r.n * src.sn;
        const bool turned = r.kind == 0 || (r.kind == 1 && a.rotate_k);
        for (uint32_t j = t; j < D; j += kGenThreads) {
            float x = Store<DT>::load1(src.data, off + j);
            if (turned && j >= a.turn.start && j < a.turn.start + a.turn.L) {
                bool first;
                const uint32_t i = turn_pair(a.turn, j - a.turn.start, &first);
                const float p = Store<DT>::load1(src.data, off + (first ? j + a.turn.half : j - a.turn.half));
                const float2 cs = turn_cos_sin(a.turn, r.b, r.s, i);
                x = rotate_own_unfused(x, p, cs.x, cs.y, first);
            }
            z[j] = x;
        }
        __syncthreads();
        if (r.kind == 0) {
            for (uint32_t j = t + a.turn.start; j < a.turn.start + a.turn.L; j += kGenThreads)
                Store<DT>::store1(src.data, off + j, z[j]);
            __syncthreads();
            continue;
        }
        const CacheRef& c = r.kind == 1 ? a.kc : a.vc;
        const int64_t page = slot / a.page_size, in_page = slot - page * a.page_size;
        char* dst = c.data + page * c.st[0] + in_page * c.st[1] + r.n * c.st[2];
        if constexpr (FMT == kFmtSame) {
            for (uint32_t j = t; j < D; j += kGenThreads) Store<DT>::store1(dst, j, z[j]);
        } else {
            const uint32_t groups = D / c.group;
            for (uint32_t g = t; g < groups; g += kGenThreads) mag[g] = 0;
            __syncthreads();
            for (uint32_t j = t; j < D; j += kGenThreads)
                atomicMax(&mag[j / c.group], __float_as_uint(finite_mag(z[j])));
            __syncthreads();
            float* sc = c.scales + page * c.sc[0] + in_page * c.sc[1] + r.n * c.sc[2];
            for (uint32_t g = t; g < groups; g += kGenThreads)
                sc[g] = group_scale<FMT>(__uint_as_float(mag[g]));
            // lanes 2i and 2i+1 share a group (groups are even)
            for (uint32_t i = t; i < D / 2; i += kGenThreads) {
                const float m = __uint_as_float(mag[2 * i / c.group]);
                const float s = group_scale<FMT>(m), inv = 1.0f / s;
                const float c0 = code_of<FMT>(z[2 * i], m, s, inv), c1 = code_of<FMT>(z[2 * i + 1], m, s, inv);
                if constexpr (FMT == kFmtInt4) {
                    dst[i] = (char)(((uint32_t)(int)c0 & 15u) | (((uint32_t)(int)c1 & 15u) << 4));
                } else {
                    const uint32_t w = pack2<FMT>(c0, c1);
                    dst[2 * i] = (char)w;
                    dst[2 * i + 1] = (char)(w >> 8);
                }
            }
        }
        __syncthreads();      // the next row overwrites z and mag
    }
}

struct CacheReadArgs {
    Rows out;
    CacheRef c;
    uint32_t N, D, S;
    uint64_t rows;            // B * S * N
    const int32_t* table;
    int64_t table_pages, table_stride;
    const int32_t* lengths;
    const int32_t* starts;
    int64_t pages, page_size;
    int32_t rotate;
    Turn turn;
    FastDiv s_div, n_div;
};

// The page and the slot within it of row s of sequence b; false when the row
// has no cached token.
__device__ __forceinline__ bool read_place(const CacheReadArgs& a, uint32_t b, uint32_t s, int64_t* page,
                                           int64_t* in_page)
{
    if ((int64_t)s >= (int64_t)a.lengths[b]) return false;
    const int64_t tok = (a.starts != nullptr ? (int64_t)a.starts[b] : 0) + s;
    if (tok < 0) return false;
    const int64_t col = tok / a.page_size;
    if (col >= a.table_pages) return false;
    *page = a.table[b * a.table_stride + col];
    *in_page = tok - col * a.page_size;
    return *page >= 0 && *page < a.pages;
}

// Lane j of a cached row as a number.
template <int DT, int FMT>
__device__ __forceinline__ float cached_lane(const CacheRef& c, const char* src, const float* sc, uint32_t j)
{
    if constexpr (FMT == kFmtSame) {
        return Store<DT>::load1(src, j);
    } else {
        float v;
        if constexpr (FMT == kFmtE4M3) {
            v = __builtin_amdgcn_cvt_f32_fp8((int)(uint8_t)src[j], 0);
        } else if constexpr (FMT == kFmtInt8) {
            v = (float)(int8_t)src[j];
        } else {
            const int w = (uint8_t)src[j / 2];
            v = (float)((j & 1u) ? (int)((uint32_t)w << 24) >> 28 : (int)((uint32_t)w << 28) >> 28);
        }
        return v * sc[j / c.group];
    }
}

template <int DT, int FMT>
__global__ void __launch_bounds__(kGenThreads) rope_cache_read_general_kernel(CacheReadArgs a)
{
    for (uint64_t row64 = blockIdx.x; row64 < a.rows; row64 += gridDim.x) {
        const uint32_t row = (uint32_t)row64;
        const uint32_t bs = fast_div(row, a.n_div);
        const uint32_t n = row - bs * a.N;
        const uint32_t b = fast_div(bs, a.s_div), s = bs - b * a.s_div.d;
        int64_t page, in_page;
        if (!read_place(a, b, s, &page, &in_page)) continue;
        const char* src = a.c.data + page * a.c.st[0] + in_page * a.c.st[1] + n * a.c.st[2];
        const float* sc = a.c.scales + page * a.c.sc[0] + in_page * a.c.sc[1] + n * a.c.sc[2];
        const int64_t off = b * a.out.sb + s * a.out.ss + n * a.out.sn;
        for (uint32_t j = threadIdx.x; j < a.D; j += kGenThreads) {
            float x = cached_lane<DT, FMT>(a.c, src, sc, j);
            if (a.rotate && j >= a.turn.start && j < a.turn.start + a.turn.L) {
                bool first;
                const uint32_t i = turn_pair(a.turn, j - a.turn.start, &first);
                const float p = cached_lane<DT, FMT>(a.c, src, sc, first ? j + a.turn.half : j - a.turn.half);
                const float2 cs = turn_cos_sin(a.turn, b, s, i);
                x = rotate_own_unfused(x, p, cs.x, cs.y, first);
            }
            Store<DT>::store1(a.out.data, off + j, x);
        }
    }
}

}  // namespace
}  // namespace rope
