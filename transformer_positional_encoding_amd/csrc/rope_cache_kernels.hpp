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
    const int64_t p = t.pos[b * t.sb + s * t.ss + axis_offset(t.ax, i)];
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

// The scale of a group whose largest finite magnitude is m: m / Q rounded to
// fp32, by the residual of its approximation (exact, and 1/Q is a correctly
// rounded constant, so the second product's sum rounds as the quotient does).
// Below 2^-100 the floor takes over.
template <int FMT>
__device__ __forceinline__ float group_scale(float m)
{
    constexpr float Q = fmt_max<FMT>(), inv = 1.0f / Q;
    const float s = m * inv;
    return m > 0.0f ? fmaxf(__builtin_fmaf(__builtin_fmaf(-s, Q, m), inv, s), 0x1p-100f) : 1.0f;
}

// 1 / s to a unit in the last place, which is all that quotient() needs.
__device__ __forceinline__ float scale_inverse(float s) { return __builtin_amdgcn_rcpf(s); }

// A float on the same side of every code and of every midpoint between two
// codes as the exact x / s, and equal to one only where x / s is. Codes and
// midpoints (t below) have at most 8 significant bits, so among fp32 numbers
// their significands are even. q is x / s within one unit in the last place
// (one Newton step on x * (1/s)) and e its residual, whose sign the fused
// multiply-add gives exactly; where e is not 0, q becomes the odd number on
// the side of q where x / s lies (q - 1 unit if it lies nearer to zero, with
// the last bit set): past no t, as a t next to it is q itself or further than
// a unit. A q that underflows has x's sign, as e does. A residual decides only
// where q is a t; x and t s are then multiples of s's last place (2^-123 or
// more, scales being 2^-100 or more) times t's (2^-10 in e4m3, 2^-1 else), so
// it is 2^-133 or more: for e4m3 and scales below 2^-93 a subnormal, which the
// code relies on being kept (as fp32 subnormals are here unless a compiler
// option asks otherwise).
__device__ __forceinline__ float quotient(float x, float s, float inv)
{
    const float q0 = x * inv;
    const float q = __builtin_fmaf(__builtin_fmaf(-q0, s, x), inv, q0);
    const float e = __builtin_fmaf(-q, s, x);
    const int32_t u = (int32_t)__float_as_uint(q);
    const int32_t nearer = ((int32_t)__float_as_uint(e) ^ u) >> 31;       // -1 or 0
    return __uint_as_float((uint32_t)(e != 0.0f ? (u + nearer) | 1 : u));
}

// The code of lane value x (as a float that the format holds) in a group of
// largest finite magnitude m and scale s. A quotient lies at most a unit or
// two in the last place over the largest code, and rounds to it.
template <int FMT>
__device__ __forceinline__ float code_of(float x, float m, float s, float inv)
{
    const float c = fminf(fmaxf(x, -m), m);        // an infinity takes the code of +-m
    float q = quotient(c, s, inv);
    if constexpr (FMT != kFmtE4M3) q = rintf(q);
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
// General kernels: any dimensions, alignment, slice and group. Writing, one wave per
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
                const float s = group_scale<FMT>(m), inv = scale_inverse(s);
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
    FastDiv s_div;
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

// A block takes a token, its waves the token's rows in turn: cos and sin are
// evaluated once a token. (A wave a row, each evaluating its own twice a pair:
// 17 sequences of up to 2947 tokens of 8 heads of 80 lanes, int4 to fp32, lanes
// [3,75) turned, 208 us; this 144, and 194 where all have 2947.)
constexpr int kGenReadThreads = 256;

template <int DT, int FMT>
__global__ void __launch_bounds__(kGenReadThreads) rope_cache_read_general_kernel(CacheReadArgs a)
{
    __shared__ float2 cs[ROPE_D_LIMIT / 2];
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t tokens = a.rows / a.N;
    for (uint64_t tok64 = blockIdx.x; tok64 < tokens; tok64 += gridDim.x) {
        const uint32_t tok = (uint32_t)tok64;
        const uint32_t b = fast_div(tok, a.s_div), s = tok - b * a.s_div.d;
        int64_t page, in_page;
        if (!read_place(a, b, s, &page, &in_page)) continue;      // the same for the whole block
        if (a.rotate) {
            __syncthreads();                                      // the rows of the token before are done
            for (uint32_t i = threadIdx.x; i < a.turn.pairs; i += kGenReadThreads) cs[i] = turn_cos_sin(a.turn, b, s, i);
            __syncthreads();
        }
        for (uint32_t n = wave; n < a.N; n += kGenReadThreads / 64) {
            const char* src = a.c.data + page * a.c.st[0] + in_page * a.c.st[1] + n * a.c.st[2];
            const float* sc = a.c.scales + page * a.c.sc[0] + in_page * a.c.sc[1] + n * a.c.sc[2];
            const int64_t off = b * a.out.sb + s * a.out.ss + n * a.out.sn;
            for (uint32_t j = lane; j < a.D; j += 64) {
                float x = cached_lane<DT, FMT>(a.c, src, sc, j);
                if (a.rotate && j >= a.turn.start && j < a.turn.start + a.turn.L) {
                    bool first;
                    const uint32_t i = turn_pair(a.turn, j - a.turn.start, &first);
                    const float p = cached_lane<DT, FMT>(a.c, src, sc, first ? j + a.turn.half : j - a.turn.half);
                    x = rotate_own_unfused(x, p, cs[i].x, cs[i].y, first);
                }
                Store<DT>::store1(a.out.data, off + j, x);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Vector kernels: rows of whole 8-lane chunks.
//
// Write. T threads of one wave share a row, a thread holding C chunks (number
// c*T + t for c < C, so that the threads of a row read consecutive 16 bytes of
// 16-bit lanes). A block takes 256/T consecutive rows of one kind (q, k or v):
// what belongs to the kind is then scalar work. It is bound by instructions as
// much as by bytes: finding a row's place costs a thread some 80 of them, a
// chunk's rotation 24 and its codes 100, so a thread takes up to three chunks
// of a row where that leaves no more lanes idle (D = 128: 8 threads of 2
// chunks; 576: 32 of 3).
// Measured on MI355X (GPU time in a graph; K and V of 3 x 2039 tokens, 8 heads
// of 128 lanes, bf16 to int8, and the (4,4096,1,576) latent to e4m3, us): 14.0
// and 15.6 (without the rotation 11.9 and 13); with 32 heads of Q beside the
// first 32.5. While the axes of the pairs were
// loaded by lane 14.6, 16.3 and 37.4; against those: one chunk a thread 21.1
// and 46; nine (the latent) 16.8; blocks of 64 or 128 threads the same within
// 0.3; one chunk a thread and waves of mixed kinds 23.7 and 20.2; several items
// a block with the next item's loads ahead 34.9 and 25.3 (its registers halve
// the waves).
// All loads of a row, and those of the chunks that hold its partners where
// these lie whole chunks away, go out first; the block's tokens' cos and sin,
// each pair of each token once, go to LDS while they are in flight; then a
// thread rotates, its group's largest magnitude is found by shuffles among the
// threads that share the group, and codes and scales are stored. q is rotated
// in place: a row lies in one wave, whose loads have all returned before its
// first store is issued.
// ---------------------------------------------------------------------------
constexpr int kVecThreads = 256;

// Global memory. Pointers that pass through an asm statement or a choice lose
// what the compiler knew of theirs, and would be accessed with the slower
// instructions for any memory.
#define ROPE_GLOBAL __attribute__((address_space(1)))
typedef ROPE_GLOBAL char gchar;

__device__ __forceinline__ gchar* as_global(const void* p) { return (gchar*)(uintptr_t)p; }
template <class V>
__device__ __forceinline__ V gload(const gchar* p)
{
    return *(const ROPE_GLOBAL V*)p;
}
template <class V>
__device__ __forceinline__ void gstore(gchar* p, V v)
{
    *(ROPE_GLOBAL V*)p = v;
}

// 8 lanes of storage type DT at p (16-byte aligned), as loaded.
template <int DT>
struct Chunk {
    static constexpr int kVecs = DT == ROPE_DTYPE_F32 ? 2 : 1;
    v4u q[kVecs];
    __device__ __forceinline__ void load(const gchar* p)
    {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) q[i] = gload<v4u>(p + 16 * i);
    }
    __device__ __forceinline__ void widen(float (&f)[8]) const
    {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            Lanes<DT> t;
            t.unpack(q[i]);
#pragma unroll
            for (int e = 0; e < 8 / kVecs; ++e) f[i * (8 / kVecs) + e] = t.v[e];
        }
    }
};

// 8 floats rounded to DT at p (16-byte aligned).
template <int DT>
__device__ __forceinline__ void store_chunk(gchar* p, const float (&f)[8])
{
    constexpr int V = Chunk<DT>::kVecs;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        Lanes<DT> t;
#pragma unroll
        for (int e = 0; e < 8 / V; ++e) t.v[e] = f[i * (8 / V) + e];
        gstore<v4u>(p + 16 * i, t.pack());
    }
}

// The largest finite magnitude of 8 lanes; *all: every lane is finite.
__device__ __forceinline__ float chunk_mag(const float (&x)[8], bool* all)
{
    float m = 0.0f, zero = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        m = fmaxf(m, fabsf(x[e]));
        zero = __builtin_fmaf(x[e], 0.0f, zero);        // NaN once a lane is not finite
    }
    *all = zero == 0.0f;
    if (!*all) {
        m = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, finite_mag(x[e]));
    }
    return m;
}

// The codes of 8 lanes at p; finite: no lane of the wave is NaN or infinite,
// so that none has to be looked at.
template <int FMT>
__device__ __forceinline__ void store_codes(gchar* p, const float (&x)[8], float m, float s, float inv, bool finite)
{
    float c[8];
    if (finite) {
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = quotient(x[e], s, inv);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = code_of<FMT>(x[e], m, s, inv);
    }
    if constexpr (FMT == kFmtE4M3) {
        int w0 = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
        w0 = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], w0, true);
        int w1 = __builtin_amdgcn_cvt_pk_fp8_f32(c[4], c[5], 0, false);
        w1 = __builtin_amdgcn_cvt_pk_fp8_f32(c[6], c[7], w1, true);
        gstore<v2u>(p, v2u{(uint32_t)w0, (uint32_t)w1});
    } else {
        // adding 1.5 * 2^23 rounds to the nearest whole number, ties to even,
        // and leaves it in the low bits
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(c[e] + 12582912.0f);
        if constexpr (FMT == kFmtInt8) {
            const auto four = [](uint32_t a, uint32_t b, uint32_t d, uint32_t f) {
                return __builtin_amdgcn_perm(__builtin_amdgcn_perm(f, d, 0x0c0c0400), __builtin_amdgcn_perm(b, a, 0x0c0c0400),
                                             0x05040100);
            };
            gstore<v2u>(p, v2u{four(w[0], w[1], w[2], w[3]), four(w[4], w[5], w[6], w[7])});
        } else {
            uint32_t v = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) v |= (w[e] & 15u) << (4 * e);
            gstore<uint32_t>(p, v);
        }
    }
}

// Where a chunk stands in the slice: its place among the block's cos and sin
// (first pair), whether it holds first lanes, its partners' chunk as a
// distance in lanes (0: within the chunk).
struct ChunkTurn {
    bool in;
    bool first;
    int32_t to_partner;
    uint32_t pair;
};

__device__ __forceinline__ ChunkTurn chunk_turn(const Turn& t, uint32_t lane0)
{
    ChunkTurn k;
    const uint32_t rel = lane0 - t.start;                // wraps below the slice
    k.in = lane0 >= t.start && rel < t.L;
    if (t.half == 1) {
        k.first = true;
        k.to_partner = 0;
        k.pair = rel / 2;
    } else {
        const uint32_t h = fast_div(k.in ? rel : 0, t.half_div);
        k.first = (h & 1u) == 0;
        k.to_partner = k.first ? (int32_t)t.half : -(int32_t)t.half;
        k.pair = (h >> 1) * t.half + rel - h * t.half;
    }
    return k;
}

// The 8 lanes of a chunk in the slice, rotated: x and its partners p (the
// chunk itself where pairs are adjacent), cos and sin of its pairs.
__device__ __forceinline__ void turn_chunk(float (&x)[8], const float (&p)[8], const ChunkTurn& k, bool adjacent,
                                           const float* cosv, const float* sinv)
{
    const float4* c4 = reinterpret_cast<const float4*>(cosv + k.pair);
    const float4* s4 = reinterpret_cast<const float4*>(sinv + k.pair);
    if (adjacent) {
        const float4 c = c4[0], s = s4[0];
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = rotate_own_unfused(a, b, cc[i], ss[i], true);
            x[2 * i + 1] = rotate_own_unfused(b, a, cc[i], ss[i], false);
        }
    } else {
        const float4 c0 = c4[0], c1 = c4[1], s0 = s4[0], s1 = s4[1];
        const float cc[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        const float ss[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = rotate_own_unfused(x[e], p[e], cc[e], ss[e], k.first);
    }
}

struct CacheWriteVecArgs : CacheWriteArgs {
    uint32_t T;               // threads per row (a power of two up to 64)
    uint32_t rows_per_block;  // 256 / T
    uint32_t blocks_q, blocks_k;   // blocks of q rows, then of k rows; the rest of v rows
    uint32_t gvk, gvv;        // chunks per scale of k and v: a power of two up to T, or 0: the whole row
    uint32_t lds_floats;      // of cos (sin follows)
    int32_t own_partner;      // C 2: a thread's two chunks hold each other's partners
    int32_t small_slots;      // slots fit 32 bits
    FastDiv t_div, nq_div, nk_div, nv_div, page_div, pairs_div;
};

// One kind of rows (scalar).
struct KindRef {
    gchar* data;
    int64_t sb, ss, sn;       // elements
    uint32_t N, D;
    FastDiv n_div;
    bool turned;
};

// An argument's value, in a scalar register. A choice between two arguments
// would otherwise become a choice between their addresses, for which the
// compiler copies all of the arguments to scratch memory.
template <class V>
__device__ __forceinline__ V held(V v)
{
    asm("" : "+s"(v));
    return v;
}

template <int DT, int FMT, int C, bool PAR>
__global__ void __launch_bounds__(kVecThreads) rope_cache_write_kernel(CacheWriteVecArgs a)
{
    extern __shared__ __attribute__((aligned(16))) float turn_lds[];   // cos of the block's tokens' pairs, then sin
    constexpr int ES = DT == ROPE_DTYPE_F32 ? 4 : 2;
    const uint32_t t = threadIdx.x, tt = t & (a.T - 1);
    const int kind = blockIdx.x < a.blocks_q ? 0 : blockIdx.x < a.blocks_q + a.blocks_k ? 1 : 2;
    const uint32_t block = blockIdx.x - (kind == 0 ? 0 : kind == 1 ? a.blocks_q : a.blocks_q + a.blocks_k);
    KindRef kr;
    if (kind == 0) kr = {as_global(held(a.q.data)), held(a.q.sb), held(a.q.ss), held(a.q.sn), held(a.Nq), held(a.Dk),
                         {held(a.nq_div.d), held(a.nq_div.mul), held(a.nq_div.shift)}, true};
    else if (kind == 1) kr = {as_global(held(a.k.data)), held(a.k.sb), held(a.k.ss), held(a.k.sn), held(a.Nk), held(a.Dk),
                              {held(a.nk_div.d), held(a.nk_div.mul), held(a.nk_div.shift)}, held(a.rotate_k) != 0};
    else kr = {as_global(held(a.v.data)), held(a.v.sb), held(a.v.ss), held(a.v.sn), held(a.Nv), held(a.Dv),
               {held(a.nv_div.d), held(a.nv_div.mul), held(a.nv_div.shift)}, false};
    const uint32_t rows = a.tokens * kr.N;
    const uint32_t row0 = block * a.rows_per_block;
    const uint32_t last = min(row0 + a.rows_per_block, rows) - 1;
    const uint32_t tok0 = fast_div(row0, kr.n_div), tok1 = fast_div(last, kr.n_div);

    // the thread's row (past the last: that one again, nothing stored)
    const uint32_t want = row0 + fast_div(t, a.t_div);
    const bool live = want <= last;
    const uint32_t row = live ? want : last;
    const uint32_t tok = fast_div(row, kr.n_div), n = row - tok * kr.N;
    const uint32_t b = fast_div(tok, a.s_div), s = tok - b * a.s_div.d;
    const int64_t slot = kind != 0 ? a.slots[b * a.slot_sb + s * a.slot_ss] : 0;
    gchar* base = kr.data + (b * kr.sb + s * kr.ss + n * kr.sn) * ES;
    Chunk<DT> own[C], par[PAR ? C : 1];
    ChunkTurn kt[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const uint32_t lane0 = (c * a.T + tt) * 8;
        const uint32_t at = lane0 < kr.D ? lane0 : 0;
        own[c].load(base + at * ES);
        kt[c] = chunk_turn(a.turn, lane0);
        kt[c].in = kt[c].in && kr.turned;
        if constexpr (PAR)
            if (kt[c].in && !(C == 2 && a.own_partner)) par[c].load(base + (int32_t)(at + kt[c].to_partner) * ES);
    }
    if (kr.turned) {
        const uint32_t entries = (tok1 - tok0 + 1) * a.turn.pairs;
        for (uint32_t e = t; e < entries; e += kVecThreads) {
            const uint32_t k = fast_div(e, a.pairs_div);
            const uint32_t be = fast_div(tok0 + k, a.s_div);
            const float2 cs = turn_cos_sin(a.turn, be, tok0 + k - be * a.s_div.d, e - k * a.turn.pairs);
            turn_lds[e] = cs.x;
            turn_lds[a.lds_floats + e] = cs.y;
        }
        __syncthreads();
    }
    const float* cosv = turn_lds + (tok - tok0) * a.turn.pairs;
    const float* sinv = cosv + a.lds_floats;
    float x[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) own[c].widen(x[c]);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (!kt[c].in) continue;
        if constexpr (PAR) {
            float p[8];
            if (C == 2 && a.own_partner) own[C - 1 - c].widen(p);
            else par[c].widen(p);
            turn_chunk(x[c], p, kt[c], false, cosv, sinv);
        } else {
            turn_chunk(x[c], x[c], kt[c], true, cosv, sinv);
        }
    }
    if (kind == 0) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (live && kt[c].in) store_chunk<DT>(base + (c * a.T + tt) * 8 * ES, x[c]);
        return;
    }
    CacheRef cr;
    const bool is_v = kind == 2;
    cr.data = is_v ? held(a.vc.data) : held(a.kc.data);
    cr.scales = is_v ? held(a.vc.scales) : held(a.kc.scales);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        cr.st[i] = is_v ? held(a.vc.st[i]) : held(a.kc.st[i]);
        cr.sc[i] = is_v ? held(a.vc.sc[i]) : held(a.kc.sc[i]);
    }
    const bool store = live && slot >= 0 && slot < a.nslots;
    int64_t page, in_page;
    if (a.small_slots) {
        const uint32_t s32 = store ? (uint32_t)slot : 0;
        const uint32_t pg = fast_div(s32, a.page_div);
        page = pg;
        in_page = s32 - pg * a.page_div.d;
    } else {
        page = slot / a.page_size;
        in_page = slot - page * a.page_size;
    }
    gchar* dst = as_global(cr.data) + (page * cr.st[0] + in_page * cr.st[1] + n * cr.st[2]);
    if constexpr (FMT == kFmtSame) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const uint32_t lane0 = (c * a.T + tt) * 8;
            if (store && lane0 < kr.D) store_chunk<DT>(dst + lane0 * ES, x[c]);
        }
    } else {
        float mag[C];
        bool fine = true;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            bool all;
            mag[c] = chunk_mag(x[c], &all);
            const bool in = (c * a.T + tt) * 8 < kr.D;
            mag[c] = in ? mag[c] : 0.0f;
            fine = fine && (all || !in);
        }
        const bool finite = __ballot(!fine) == 0;
        const uint32_t gv = is_v ? held(a.gvv) : held(a.gvk);
        if (C > 1 && gv == 0) {
            float m = mag[0];
#pragma unroll
            for (int c = 1; c < C; ++c) m = fmaxf(m, mag[c]);
#pragma unroll
            for (int c = 0; c < C; ++c) mag[c] = m;
        }
        const uint32_t width = gv == 0 ? a.T : gv;
        for (uint32_t d = 1; d < width; d <<= 1)
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (c == 0 || gv != 0) mag[c] = fmaxf(mag[c], __shfl_xor(mag[c], (int)d));
        gchar* sc = as_global(cr.scales) + (page * cr.sc[0] + in_page * cr.sc[1] + n * cr.sc[2]) * 4;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const uint32_t chunk = c * a.T + tt;
            if (!store || chunk * 8 >= kr.D) continue;
            const float m = gv != 0 ? mag[c] : mag[0];
            const float sv = group_scale<FMT>(m), inv = scale_inverse(sv);
            store_codes<FMT>(dst + (FMT == kFmtInt4 ? chunk * 4 : chunk * 8), x[c], m, sv, inv, finite);
            if (gv == 0) {
                if (chunk == 0) gstore<float>(sc, sv);
            } else if ((chunk & (gv - 1)) == 0) {
                gstore<float>(sc + chunk / gv * 4, sv);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Read, vector form: bound by the bytes it moves. A token's N rows are N * D/8
// chunks. A wave takes a whole token, so that its sequence, page and addresses
// are scalar work, where the token fills its passes of 64 chunks (below);
// otherwise 512 consecutive chunks of the output go to a block, two a thread
// whose loads go out together, each finding its token.
// Measured on MI355X (e4m3 to bf16, 134 million lanes and, in brackets, 8
// million; us by waves and by blocks, tokens of
//   chunks    not turned               32 pairs turned          64 pairs turned
//   16        258, 99 (18, 8.1)        468, 203 (34, 17)        470, 284 (33, 24)
//   48        119, 101 (9.8, 8.2)      184, 159 (15, 13)        184, 180 (15, 15)
//   56        105, 102 (9.2, 8.2)      165, 156 (14, 13)
//   64        93, 99 (8.8, 8.2)        148, 145 (13, 12)        148, 163 (13, 14)
//   72        124, 100 (10, 8.2)       176, 145 (16, 12)        184, 163 (16, 13)
//   96        106, 101 (9.4, 8.2)      159, 143 (15, 12)        160, 158 (15, 13)
//   112       95, 100 (9.0, 8.1)       142, 143 (14, 12)        142, 157 (14, 13)
//   128       78, 99 (7.8, 8.2)        106, 140 (12, 12)        107, 144 (12, 12)
//   144       84, 101 (8.0, 8.2)       117, 142 (12, 12)        117, 151 (12, 13)
// and no further apart with the other formats.) Blocks of one chunk a thread 121
// where two take 99, of four 100.
// 12 sequences of up to 16384 tokens, 8 heads of 128 lanes, e4m3 to bf16, take
// 88 us (5.2 TB/s); 3 x 6135 tokens of int8, 14.5; 5 x 3257 tokens of 4 heads,
// int4 to fp16, 8.3, and with 32 pairs turned by fp32 cos and sin, evaluated in
// double by their blocks, 11.8.
// ---------------------------------------------------------------------------
constexpr int kReadChunks = 2;

struct CacheReadVecArgs : CacheReadArgs {
    uint32_t chunks;          // of a row
    uint32_t token_chunks;    // of a token: N * chunks
    uint32_t tokens;
    uint32_t group_shift;     // log2 of the lanes per scale / 8, or 31: one scale a row
    int32_t small_tokens;     // a block table's token numbers fit 31 bits
    FastDiv chunk_div, token_div, page_div, pairs_div;
};

// 8 codes as numbers (not yet scaled).
template <int DT, int FMT>
struct CodeChunk {
    using Raw = typename std::conditional<FMT == kFmtSame, Chunk<DT>,
                                          typename std::conditional<FMT == kFmtInt4, uint32_t, v2u>::type>::type;
    Raw q;
    float s;
    __device__ __forceinline__ void load(const CacheReadVecArgs& a, const gchar* src, const gchar* sc, uint32_t chunk)
    {
        if constexpr (FMT == kFmtSame) {
            q.load(src + chunk * (DT == ROPE_DTYPE_F32 ? 32 : 16));
        } else {
            q = gload<Raw>(src + chunk * (FMT == kFmtInt4 ? 4 : 8));
            s = gload<float>(sc + (a.group_shift == 31 ? 0 : chunk >> a.group_shift) * 4);
        }
    }
    __device__ __forceinline__ void widen(float (&f)[8]) const
    {
        if constexpr (FMT == kFmtSame) {
            q.widen(f);
        } else if constexpr (FMT == kFmtE4M3) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[i], false);
                const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[i], true);
                f[4 * i] = lo.x * s;
                f[4 * i + 1] = lo.y * s;
                f[4 * i + 2] = hi.x * s;
                f[4 * i + 3] = hi.y * s;
            }
        } else if constexpr (FMT == kFmtInt8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = (float)((int)(q[e / 4] << (24 - 8 * (e % 4))) >> 24) * s;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = (float)((int)(q << (28 - 4 * e)) >> 28) * s;
        }
    }
};

// As read_place, with the token's number in 32 bits where it fits.
__device__ __forceinline__ bool read_place32(const CacheReadVecArgs& a, uint32_t b, uint32_t s, int64_t* page,
                                             int64_t* in_page)
{
    if (!a.small_tokens) return read_place(a, b, s, page, in_page);
    const int32_t len = a.lengths[b], start = a.starts != nullptr ? a.starts[b] : 0;
    const int64_t tok64 = (int64_t)start + s;
    const bool ok = (int64_t)s < (int64_t)len && tok64 >= 0 && tok64 < (int64_t)0x7FFFFFFF;
    const uint32_t tok = ok ? (uint32_t)tok64 : 0;
    const uint32_t col = fast_div(tok, a.page_div);
    if (!ok || (int64_t)col >= a.table_pages) return false;
    *page = a.table[b * a.table_stride + col];
    *in_page = tok - col * a.page_div.d;
    return *page >= 0 && *page < a.pages;
}

template <int DT, int FMT, bool ROT>
__device__ __forceinline__ void read_chunk(const CacheReadVecArgs& a, const gchar* src, const gchar* sc, gchar* dst,
                                           uint32_t chunk, const float* cosv, const float* sinv)
{
    constexpr int ES = DT == ROPE_DTYPE_F32 ? 4 : 2;
    CodeChunk<DT, FMT> own, par;
    own.load(a, src, sc, chunk);
    float x[8];
    if constexpr (ROT) {
        const ChunkTurn k = chunk_turn(a.turn, chunk * 8);
        const bool adjacent = a.turn.half == 1;
        if (k.in && !adjacent) par.load(a, src, sc, (uint32_t)((int32_t)(chunk * 8) + k.to_partner) / 8);
        own.widen(x);
        if (k.in) {
            float p[8];
            if (adjacent) {
#pragma unroll
                for (int e = 0; e < 8; ++e) p[e] = 0.0f;
            } else {
                par.widen(p);
            }
            turn_chunk(x, p, k, adjacent, cosv, sinv);
        }
    } else {
        own.widen(x);
    }
    store_chunk<DT>(dst + chunk * 8 * ES, x);
}

// As read_place32 without a branch: where there is no cached token, page and
// slot 0, which may be read.
__device__ __forceinline__ bool read_place_always(const CacheReadVecArgs& a, uint32_t b, uint32_t s, int64_t* page,
                                                  int64_t* in_page)
{
    const int32_t len = a.lengths[b], start = a.starts != nullptr ? a.starts[b] : 0;
    const int64_t tok64 = (int64_t)start + s;
    bool ok = (int64_t)s < (int64_t)len && tok64 >= 0;
    int64_t col, in;
    if (a.small_tokens) {
        ok = ok && tok64 < (int64_t)0x7FFFFFFF;
        const uint32_t tok = ok ? (uint32_t)tok64 : 0;
        const uint32_t c32 = fast_div(tok, a.page_div);
        col = c32;
        in = tok - c32 * a.page_div.d;
    } else {
        const int64_t tok = ok ? tok64 : 0;
        col = tok / a.page_size;
        in = tok - col * a.page_size;
    }
    ok = ok && col < a.table_pages;
    const int64_t pg = a.table[b * a.table_stride + min(col, a.table_pages - 1)];
    ok = ok && pg >= 0 && pg < a.pages;
    *page = ok ? pg : 0;
    *in_page = ok ? in : 0;
    return ok;
}

template <int DT, int FMT, bool ROT>
__global__ void __launch_bounds__(kVecThreads) rope_cache_read_kernel(CacheReadVecArgs a)
{
    constexpr int ES = DT == ROPE_DTYPE_F32 ? 4 : 2;
    constexpr int U = kReadChunks;
    extern __shared__ __attribute__((aligned(16))) float turn_lds[];   // ROT: cos of the block's tokens' pairs, then sin
    const uint32_t i0 = blockIdx.x * (U * kVecThreads);
    const uint32_t total = a.tokens * a.token_chunks;
    const uint32_t tok0 = fast_div(i0, a.token_div);
    CodeChunk<DT, FMT> own[U], par[ROT ? U : 1];
    ChunkTurn kt[ROT ? U : 1];
    gchar* dst[U];
    uint32_t at[U];
    bool ok[U];
    const bool adjacent = a.turn.half == 1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t want = i0 + u * kVecThreads + threadIdx.x;
        const uint32_t i = min(want, total - 1);
        const uint32_t tok = fast_div(i, a.token_div);
        const uint32_t c = i - tok * a.token_chunks;
        const uint32_t n = fast_div(c, a.chunk_div), chunk = c - n * a.chunks;
        const uint32_t b = fast_div(tok, a.s_div), s = tok - b * a.s_div.d;
        int64_t page, in_page;
        ok[u] = read_place_always(a, b, s, &page, &in_page) && want < total;
        const gchar* src = as_global(a.c.data) + page * a.c.st[0] + in_page * a.c.st[1] + n * a.c.st[2];
        const gchar* sc = as_global(a.c.scales + page * a.c.sc[0] + in_page * a.c.sc[1] + n * a.c.sc[2]);
        own[u].load(a, src, sc, chunk);
        if constexpr (ROT) {
            kt[u] = chunk_turn(a.turn, chunk * 8);
            const int32_t away = kt[u].in && !adjacent ? kt[u].to_partner : 0;
            par[u].load(a, src, sc, (uint32_t)((int32_t)(chunk * 8) + away) / 8);
        }
        dst[u] = as_global(a.out.data) + (b * a.out.sb + s * a.out.ss + n * a.out.sn) * ES + chunk * 8 * ES;
        at[u] = (tok - tok0) * a.turn.pairs;
    }
    float* sinv = turn_lds;
    if constexpr (ROT) {
        const uint32_t tok1 = fast_div(min(i0 + U * kVecThreads, total) - 1, a.token_div);
        const uint32_t entries = (tok1 - tok0 + 1) * a.turn.pairs;
        sinv += entries;
        for (uint32_t e = threadIdx.x; e < entries; e += kVecThreads) {
            const uint32_t k = fast_div(e, a.pairs_div);
            const uint32_t be = fast_div(tok0 + k, a.s_div);
            const float2 cs = turn_cos_sin(a.turn, be, tok0 + k - be * a.s_div.d, e - k * a.turn.pairs);
            turn_lds[e] = cs.x;
            sinv[e] = cs.y;
        }
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float x[8];
        own[u].widen(x);
        if constexpr (ROT) {
            if (kt[u].in) {
                float p[8];
                par[u].widen(p);
                turn_chunk(x, p, kt[u], adjacent, turn_lds + at[u], sinv + at[u]);
            }
        }
        if (ok[u]) store_chunk<DT>(dst[u], x);
    }
}

template <int DT, int FMT, bool ROT>
__global__ void __launch_bounds__(kVecThreads) rope_cache_read_wave_kernel(CacheReadVecArgs a)
{
    constexpr int ES = DT == ROPE_DTYPE_F32 ? 4 : 2;
    __shared__ __attribute__((aligned(16))) float turn_lds[ROT ? 4 * ROPE_D_LIMIT : 4];
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t tok = blockIdx.x * 4 + wave;
    if (tok >= a.tokens) return;
    const uint32_t b = fast_div(tok, a.s_div), s = tok - b * a.s_div.d;
    int64_t page, in_page;
    if (!read_place32(a, b, s, &page, &in_page)) return;
    const float* cosv = nullptr;
    const float* sinv = nullptr;
    if constexpr (ROT) {
        // the token's cos and sin, by the wave for itself
        float* mine = turn_lds + wave * ROPE_D_LIMIT;
        for (uint32_t e = lane; e < a.turn.pairs; e += 64) {
            const float2 cs = turn_cos_sin(a.turn, b, s, e);
            mine[e] = cs.x;
            mine[a.turn.pairs + e] = cs.y;
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        cosv = mine;
        sinv = mine + a.turn.pairs;
    }
    const gchar* src = as_global(a.c.data) + page * a.c.st[0] + in_page * a.c.st[1];
    const gchar* sc = as_global(a.c.scales + page * a.c.sc[0] + in_page * a.c.sc[1]);
    gchar* dst = as_global(a.out.data) + (b * a.out.sb + s * a.out.ss) * ES;
#pragma unroll 2
    for (uint32_t c = lane; c < a.token_chunks; c += 64) {
        const uint32_t n = fast_div(c, a.chunk_div), chunk = c - n * a.chunks;
        read_chunk<DT, FMT, ROT>(a, src + n * a.c.st[2], sc + n * a.c.sc[2] * 4, dst + n * a.out.sn * ES, chunk, cosv, sinv);
    }
}

}  // namespace
}  // namespace rope
