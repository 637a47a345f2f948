// rope_norm_kernels.hpp -- RMS norms of the heads of Q and K with the position
// rotation in the same pass, forward and backward.
// Included by rope_norm.hip, next to the host code that launches them.
//
// Mathematics, for a row x of D lanes, its weight w and its token's rotation R:
//   r = 1 / sqrt(mean(x^2) + eps),  n = r x,  y = R (n w)
//   backward, with g = R^T dy:
//   dw = sum over rows of g n,  dx = r (g w - n mean(g w n))
// All in fp32 (x^2 summed, y, dx and dw rounded once, when stored). The sum of
// g w x does not need r, so that one reduction gives both sums of a row.
#pragma once

#include "rope_cache_kernels.hpp"

namespace rope {
namespace {

struct NormArgs {
    Rows x[2], y[2], dy[2];   // of Q and of K
    const void* w[2];         // NULL: ones
    uint32_t N[2];
    uint32_t D, tokens, S;
    int32_t wdt;
    float eps, inv_d;
    int32_t rotate;
    float* part;              // backward: blocks x 2 x D sums, or NULL
    Turn turn;
    FastDiv s_div;
};

__device__ __forceinline__ float norm_weight(const NormArgs& a, int kind, uint32_t j)
{
    const void* w = a.w[kind];
    if (w == nullptr) return 1.0f;
    switch (a.wdt) {
    case ROPE_DTYPE_F32: return Store<ROPE_DTYPE_F32>::load1(w, j);
    case ROPE_DTYPE_F16: return Store<ROPE_DTYPE_F16>::load1(w, j);
    default: return Store<ROPE_DTYPE_BF16>::load1(w, j);
    }
}

// Pairs that lie beside each other, turned back.
__device__ __forceinline__ void turn_back_adjacent(float (&g)[8], const ChunkTurn& k, const float* cosv, const float* sinv)
{
    const float4 c = *reinterpret_cast<const float4*>(cosv + k.pair), s = *reinterpret_cast<const float4*>(sinv + k.pair);
    const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float p = g[2 * i], q = g[2 * i + 1];
        g[2 * i] = rotate_own_unfused(p, q, cc[i], sn[i], false);
        g[2 * i + 1] = rotate_own_unfused(q, p, cc[i], sn[i], true);
    }
}

// The sum over the lanes of a wave that differ in the bits below `width` (a
// power of two), the same in all of them: by exchanges on the vector unit. (A
// lane of the mirrored half row holds what the lane 4 or 8 away does, once
// quads or eights are summed.)
__device__ __forceinline__ float lanes_sum(float v, uint32_t width)
{
    const auto dpp = [](float x, auto ctrl) {
        return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(x), decltype(ctrl)::value, 0xF, 0xF, true));
    };
    if (width > 1) v += dpp(v, std::integral_constant<int, 0xB1>{});       // lane ^ 1
    if (width > 2) v += dpp(v, std::integral_constant<int, 0x4E>{});       // lane ^ 2
    if (width > 4) v += dpp(v, std::integral_constant<int, 0x141>{});      // mirrored eights
    if (width > 8) v += dpp(v, std::integral_constant<int, 0x140>{});      // mirrored sixteens
    if (width > 16) {
        const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    }
    if (width > 32) {
        const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    }
    return v;
}

// ---------------------------------------------------------------------------
// General kernels: any dimensions, alignment and slice. A block takes a token,
// each of its waves every fourth of the token's rows, with the next one's lanes
// on the way; cos and sin are evaluated once a token, and a row stands in the
// wave's part of LDS for its partners' sake. Single lanes, and a row a wave: the
// instructions bound it. 2 x 2000 tokens of 36 heads: of 36 lanes 35 us (0.6
// TB/s), of 128 with 20 of them rotated 53 (1.4); forward and backward of 4 x
// 2000 tokens of 40 heads of 96, 24 rotated, 308 us (1 TB/s).
// ---------------------------------------------------------------------------
constexpr int kNormThreads = 256;
constexpr int kNormWaves = kNormThreads / 64;
// NL: lanes of a row that a thread takes at most, for rows of up to 256 and of
// any number.
constexpr int kNormFewLanes = 4, kNormLanes = ROPE_D_LIMIT / 64;

// cos and sin of a token's pairs, once the rows of the token before are done.
__device__ __forceinline__ void norm_turns(const NormArgs& a, uint32_t b, uint32_t s, float2* cs)
{
    if (!a.rotate) return;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < a.turn.pairs; i += kNormThreads) cs[i] = turn_cos_sin(a.turn, b, s, i);
    __syncthreads();
}

// What a wave writes to its part of LDS is there for its other lanes.
__device__ __forceinline__ void norm_wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// What a thread's lanes keep from row to row: where their pairs' partners and
// angles are, and the weights of a kind.
template <int NL>
struct NormLanes {
    int32_t partner[NL];                  // -1: not turned
    uint32_t pair[NL];
    bool first[NL];
    float w[NL];
    __device__ __forceinline__ NormLanes(const NormArgs& a, uint32_t lane)
    {
#pragma unroll
        for (int k = 0; k < NL; ++k) {
            const uint32_t j = k * 64 + lane;
            partner[k] = -1;
            pair[k] = 0;
            first[k] = false;
            if (a.rotate && j >= a.turn.start && j < a.turn.start + a.turn.L && j < a.D) {
                pair[k] = turn_pair(a.turn, j - a.turn.start, &first[k]);
                partner[k] = (int32_t)(first[k] ? j + a.turn.half : j - a.turn.half);
            }
        }
    }
    __device__ __forceinline__ void weights(const NormArgs& a, int kind, uint32_t lane)
    {
#pragma unroll
        for (int k = 0; k < NL; ++k) w[k] = k * 64 + lane < a.D ? norm_weight(a, kind, k * 64 + lane) : 0.0f;
    }
    // Number k of them of a row that stands in LDS, its pair turned.
    __device__ __forceinline__ float turned(int k, uint32_t lane, const float* z, const float2* cs, bool back) const
    {
        float v = z[k * 64 + lane];
        if (partner[k] >= 0) v = rotate_own_unfused(v, z[partner[k]], cs[pair[k]].x, cs[pair[k]].y, first[k] != back);
        return v;
    }
};

// A thread's lanes of a row.
template <int DT, int NL>
__device__ __forceinline__ void norm_row_lanes(const NormArgs& a, const Rows& x, uint32_t b, uint32_t s, uint32_t n, uint32_t lane,
                                               float (&v)[NL])
{
    const int64_t row = b * x.sb + s * x.ss + n * x.sn;
#pragma unroll
    for (int k = 0; k < NL; ++k) {
        if (k * 64 >= a.D) break;
        const uint32_t j = k * 64 + lane;
        v[k] = j < a.D ? Store<DT>::load1(x.data, row + j) : 0.0f;
    }
}

template <int DT, int NL>
__global__ void __launch_bounds__(kNormThreads) rope_norm_fwd_general_kernel(NormArgs a)
{
    __shared__ float2 cs[ROPE_D_LIMIT / 2];
    __shared__ float rows[kNormWaves][ROPE_D_LIMIT];
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float* z = rows[wave];
    NormLanes<NL> own(a, lane);
    for (uint32_t tok = blockIdx.x; tok < a.tokens; tok += gridDim.x) {
        const uint32_t b = fast_div(tok, a.s_div), s = tok - b * a.S;
        norm_turns(a, b, s, cs);
        for (int kind = 0; kind < 2; ++kind) {
            const Rows& y = a.y[kind];
            float next[NL];
            if (wave < a.N[kind]) norm_row_lanes<DT, NL>(a, a.x[kind], b, s, wave, lane, next);
            own.weights(a, kind, lane);
            for (uint32_t n = wave; n < a.N[kind]; n += kNormWaves) {
                float v[NL], ss = 0.0f;
#pragma unroll
                for (int k = 0; k < NL; ++k) {
                    if (k * 64 >= a.D) break;
                    v[k] = next[k];
                    ss = __builtin_fmaf(v[k], v[k], ss);
                }
                if (n + kNormWaves < a.N[kind]) norm_row_lanes<DT, NL>(a, a.x[kind], b, s, n + kNormWaves, lane, next);
                const float r = rsqrtf(__builtin_fmaf(lanes_sum(ss, 64), a.inv_d, a.eps));
                norm_wave_sync();                  // the row before is done
#pragma unroll
                for (int k = 0; k < NL; ++k) {
                    if (k * 64 >= a.D) break;
                    const uint32_t j = k * 64 + lane;
                    if (j < a.D) z[j] = v[k] * r * own.w[k];
                }
                norm_wave_sync();
                const int64_t row = b * y.sb + s * y.ss + n * y.sn;
#pragma unroll
                for (int k = 0; k < NL; ++k) {
                    if (k * 64 >= a.D) break;
                    const uint32_t j = k * 64 + lane;
                    if (j < a.D) Store<DT>::store1(y.data, row + j, own.turned(k, lane, z, cs, false));
                }
            }
        }
    }
}

template <int DT, int NL>
__global__ void __launch_bounds__(kNormThreads) rope_norm_bwd_general_kernel(NormArgs a)
{
    __shared__ float2 cs[ROPE_D_LIMIT / 2];
    __shared__ float rows[kNormWaves][ROPE_D_LIMIT];
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float* z = rows[wave];
    NormLanes<NL> own(a, lane);
    for (int kind = 0; kind < 2; ++kind) {
        const Rows& y = a.y[kind];
        float dw[NL] = {};
        own.weights(a, kind, lane);
        for (uint32_t tok = blockIdx.x; tok < a.tokens; tok += gridDim.x) {
            if (a.N[kind] == 0) break;
            const uint32_t b = fast_div(tok, a.s_div), s = tok - b * a.S;
            norm_turns(a, b, s, cs);
            float next[NL], up[NL];
            if (wave < a.N[kind]) {
                norm_row_lanes<DT, NL>(a, a.x[kind], b, s, wave, lane, next);
                norm_row_lanes<DT, NL>(a, a.dy[kind], b, s, wave, lane, up);
            }
            for (uint32_t n = wave; n < a.N[kind]; n += kNormWaves) {
                float v[NL], g[NL], ss = 0.0f, dot = 0.0f;
                norm_wave_sync();                  // the row before is done
#pragma unroll
                for (int k = 0; k < NL; ++k) {
                    if (k * 64 >= a.D) break;
                    v[k] = next[k];
                    if (k * 64 + lane < a.D) z[k * 64 + lane] = up[k];
                }
                if (n + kNormWaves < a.N[kind]) {
                    norm_row_lanes<DT, NL>(a, a.x[kind], b, s, n + kNormWaves, lane, next);
                    norm_row_lanes<DT, NL>(a, a.dy[kind], b, s, n + kNormWaves, lane, up);
                }
                norm_wave_sync();
#pragma unroll
                for (int k = 0; k < NL; ++k) {
                    if (k * 64 >= a.D) break;
                    const uint32_t j = k * 64 + lane;
                    g[k] = 0.0f;
                    if (j >= a.D) continue;
                    g[k] = own.turned(k, lane, z, cs, true);
                    ss = __builtin_fmaf(v[k], v[k], ss);
                    dot = __builtin_fmaf(g[k] * own.w[k], v[k], dot);
                }
                const float r = rsqrtf(__builtin_fmaf(lanes_sum(ss, 64), a.inv_d, a.eps));
                const float m = lanes_sum(dot, 64) * r * a.inv_d;
                const int64_t row = b * y.sb + s * y.ss + n * y.sn;
#pragma unroll
                for (int k = 0; k < NL; ++k) {
                    if (k * 64 >= a.D) break;
                    const uint32_t j = k * 64 + lane;
                    if (j >= a.D) continue;
                    const float nj = v[k] * r;
                    dw[k] = __builtin_fmaf(g[k], nj, dw[k]);
                    Store<DT>::store1(y.data, row + j, r * (g[k] * own.w[k] - nj * m));
                }
            }
        }
        if (a.part == nullptr) continue;
        norm_wave_sync();
#pragma unroll
        for (int k = 0; k < NL; ++k)
            if (k * 64 + lane < a.D) z[k * 64 + lane] = dw[k];
        __syncthreads();
        for (uint32_t j = threadIdx.x; j < a.D; j += kNormThreads) {
            float sum = 0.0f;
            for (int w = 0; w < kNormWaves; ++w) sum += rows[w][j];
            a.part[((uint64_t)blockIdx.x * 2 + kind) * a.D + j] = sum;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Vector kernels: rows of whole 8-lane chunks. T threads of one wave share a
// row, a thread holding C chunks (number c * T + t), as in the cache's write.
// A block takes a few tokens: their cos and sin go to LDS, each pair of a token
// evaluated once for all of its heads while the first rows are loaded; then the
// rows of Q, then those of K, so that a thread's weights stay in registers for
// all rows of a kind. Partners that lie whole chunks away are loaded with the
// row (from the cache's line that the row's own thread loads) and normalised
// again, unless the thread has them. Bound by memory: forward, 2 x 8191 tokens
// of 36 heads of 128 lanes, 302 MB: 58 us (5.2 TB/s); backward, 4 x 4096 of 40
// heads, 503 MB: 115 us (4.4).
// ---------------------------------------------------------------------------
// Where a chunk's partners are: in the chunk (or it is not turned), in a chunk
// that is loaded, in the thread's other chunk (C 2).
constexpr int kParNear = 0, kParLoad = 1, kParOwn = 2;

struct NormVecArgs : NormArgs {
    uint32_t T;                // threads per row
    uint32_t rows_per_block;   // 256 / T
    uint32_t tokens_per_block;
    uint32_t groups;           // of tokens_per_block tokens
    uint32_t splits;           // blocks that share a token's heads (tokens_per_block is 1 then)
    uint32_t lds_floats;       // of cos (sin follows)
    FastDiv t_div, n_div[2], pairs_div, splits_div;
};

// 8 lanes of a weight.
__device__ __forceinline__ void norm_weight8(const NormVecArgs& a, int kind, uint32_t j, float (&w)[8])
{
    const gchar* p = as_global(a.w[kind]);
    if (a.w[kind] == nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.0f;
    } else if (a.wdt == ROPE_DTYPE_F32) {
        Chunk<ROPE_DTYPE_F32> c;
        c.load(p + j * 4);
        c.widen(w);
    } else {
        Chunk<ROPE_DTYPE_F16> c;
        c.load(p + j * 2);
        if (a.wdt == ROPE_DTYPE_F16) {
            c.widen(w);
        } else {
            Chunk<ROPE_DTYPE_BF16> b;
            b.q[0] = c.q[0];
            b.widen(w);
        }
    }
}

// The weights of a thread's chunks, and of their partners' where these are
// loaded.
template <int C, int PAR>
struct NormWeights {
    float own[C][8], par[PAR == kParLoad ? C : 1][8];
    __device__ __forceinline__ void load(const NormVecArgs& a, int kind, const ChunkTurn (&k)[C], uint32_t tt)
    {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const uint32_t lane0 = (c * a.T + tt) * 8, at = lane0 < a.D ? lane0 : 0;      // (past the row: not stored)
            norm_weight8(a, kind, at, own[c]);
            if constexpr (PAR == kParLoad) norm_weight8(a, kind, k[c].in ? at + k[c].to_partner : at, par[c]);
        }
    }
};

// cos and sin of n tokens' pairs from token tok0 on, to LDS.
__device__ __forceinline__ void norm_turn_table(const NormVecArgs& a, uint32_t tok0, uint32_t n, float* lds)
{
    const uint32_t entries = n * a.turn.pairs;
    for (uint32_t i = threadIdx.x; i < entries; i += kNormThreads) {
        const uint32_t k = fast_div(i, a.pairs_div);
        const uint32_t b = fast_div(tok0 + k, a.s_div);
        const float2 cs = turn_cos_sin(a.turn, b, tok0 + k - b * a.S, i - k * a.turn.pairs);
        lds[i] = cs.x;
        lds[a.lds_floats + i] = cs.y;
    }
}

// The row of a thread among those of a kind: token tok0 + k, head n.
struct NormRow {
    uint32_t k, b, s, n;
};
__device__ __forceinline__ NormRow norm_row(const NormVecArgs& a, int kind, uint32_t tok0, uint32_t n0, uint32_t it)
{
    NormRow r;
    r.k = a.splits > 1 ? 0 : fast_div(it, a.n_div[kind]);
    r.n = n0 + it - r.k * a.N[kind];
    const uint32_t tok = tok0 + r.k;
    r.b = fast_div(tok, a.s_div);
    r.s = tok - r.b * a.S;
    return r;
}

template <int DT, int C, int PAR>
__global__ void __launch_bounds__(kNormThreads) rope_norm_fwd_kernel(NormVecArgs a)
{
    extern __shared__ __attribute__((aligned(16))) float norm_lds[];
    constexpr int ES = DT == ROPE_DTYPE_F32 ? 4 : 2;
    const uint32_t t = threadIdx.x, tt = t & (a.T - 1), r0 = fast_div(t, a.t_div);
    const uint32_t group = fast_div(blockIdx.x, a.splits_div), split = blockIdx.x - group * a.splits;
    const uint32_t tok0 = group * a.tokens_per_block, ntok = min(a.tokens_per_block, a.tokens - tok0);
    ChunkTurn kt[C];
#pragma unroll
    for (int c = 0; c < C; ++c) kt[c] = chunk_turn(a.turn, (c * a.T + tt) * 8);
    bool table = a.turn.L == 0;
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
        const uint32_t per = (a.N[kind] + a.splits - 1) / a.splits;
        const uint32_t n0 = min(a.N[kind], split * per), n1 = min(a.N[kind], n0 + per);
        const uint32_t rows = ntok * (n1 - n0);
        if (rows == 0) continue;
        const gchar* const xd = as_global(a.x[kind].data);
        gchar* const yd = as_global(a.y[kind].data);
        Chunk<DT> own[C], par[PAR == kParLoad ? C : 1];
        // a row's loads go out ahead of the row before it, the first ones' ahead
        // of the table (threads without a row: the last one's)
        const auto load = [&](uint32_t it) {
            const NormRow r = norm_row(a, kind, tok0, n0, min(it, rows - 1));
            const gchar* src = xd + (r.b * a.x[kind].sb + r.s * a.x[kind].ss + r.n * a.x[kind].sn) * ES;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const uint32_t lane0 = (c * a.T + tt) * 8, at = lane0 < a.D ? lane0 : 0;
                own[c].load(src + at * ES);
                if constexpr (PAR == kParLoad)
                    if (kt[c].in) par[c].load(src + (int32_t)(at + kt[c].to_partner) * ES);
            }
            return r;
        };
        NormRow next = load(r0);
        NormWeights<C, PAR> w;
        w.load(a, kind, kt, tt);
        if (!table) {
            norm_turn_table(a, tok0, ntok, norm_lds);
            __syncthreads();
            table = true;
        }
        for (uint32_t it = r0; it < rows; it += a.rows_per_block) {
            const NormRow r = next;
            gchar* dst = yd + (r.b * a.y[kind].sb + r.s * a.y[kind].ss + r.n * a.y[kind].sn) * ES;
            float x[C][8], p[PAR == kParLoad ? C : 1][8], ss = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                own[c].widen(x[c]);
                if constexpr (PAR == kParLoad) par[c].widen(p[c]);
                float sum = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(x[c][e], x[c][e], sum);
                ss += (c * a.T + tt) * 8 < a.D ? sum : 0.0f;
            }
            next = load(it + a.rows_per_block);
            const float inv = rsqrtf(__builtin_fmaf(lanes_sum(ss, a.T), a.inv_d, a.eps));
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) x[c][e] = x[c][e] * inv * w.own[c][e];
            const float* cosv = norm_lds + r.k * a.turn.pairs;
            const float* sinv = cosv + a.lds_floats;
            if constexpr (PAR == kParOwn) {
                float first[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) first[e] = x[0][e];
                turn_chunk(x[0], x[C - 1], kt[0], false, cosv, sinv);
                turn_chunk(x[C - 1], first, kt[C - 1], false, cosv, sinv);
            } else {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    if (!kt[c].in) continue;
                    if constexpr (PAR == kParLoad) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) p[c][e] = p[c][e] * inv * w.par[c][e];
                        turn_chunk(x[c], p[c], kt[c], false, cosv, sinv);
                    } else {
                        turn_chunk(x[c], x[c], kt[c], true, cosv, sinv);
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const uint32_t lane0 = (c * a.T + tt) * 8;
                if (lane0 < a.D) store_chunk<DT>(dst + lane0 * ES, x[c]);
            }
        }
    }
}

// Backward: blocks take groups of tokens in turn; a thread sums its lanes' part
// of the weight's gradient over all of its rows, and the block leaves one sum
// per lane (lanes of one chunk lie in threads T apart).
template <int DT, int C, int PAR>
__global__ void __launch_bounds__(kNormThreads, C == 1 ? 4 : 2) rope_norm_bwd_kernel(NormVecArgs a)
{
    extern __shared__ __attribute__((aligned(16))) float norm_lds[];
    constexpr int ES = DT == ROPE_DTYPE_F32 ? 4 : 2;
    const uint32_t t = threadIdx.x, tt = t & (a.T - 1), r0 = fast_div(t, a.t_div);
    ChunkTurn kt[C];
#pragma unroll
    for (int c = 0; c < C; ++c) kt[c] = chunk_turn(a.turn, (c * a.T + tt) * 8);
    float dw[2][C][8] = {};
    for (uint32_t group = blockIdx.x; group < a.groups; group += gridDim.x) {
        const uint32_t tok0 = group * a.tokens_per_block, ntok = min(a.tokens_per_block, a.tokens - tok0);
        if (a.turn.L > 0) {
            __syncthreads();                       // the rows of the group before are done
            norm_turn_table(a, tok0, ntok, norm_lds);
            __syncthreads();
        }
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
            const uint32_t rows = ntok * a.N[kind];
            if (rows == 0) continue;
            float w[C][8];
#pragma unroll
            for (int c = 0; c < C; ++c) norm_weight8(a, kind, (c * a.T + tt) * 8 < a.D ? (c * a.T + tt) * 8 : 0, w[c]);
            const gchar* const xd = as_global(a.x[kind].data);
            const gchar* const gd = as_global(a.dy[kind].data);
            gchar* const yd = as_global(a.y[kind].data);
            Chunk<DT> own[C], up[C], par[PAR == kParLoad ? C : 1];
            const auto load = [&](uint32_t it) {   // as in the forward
                const NormRow r = norm_row(a, kind, tok0, 0, min(it, rows - 1));
                const gchar* src = xd + (r.b * a.x[kind].sb + r.s * a.x[kind].ss + r.n * a.x[kind].sn) * ES;
                const gchar* grad = gd + (r.b * a.dy[kind].sb + r.s * a.dy[kind].ss + r.n * a.dy[kind].sn) * ES;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const uint32_t lane0 = (c * a.T + tt) * 8, at = lane0 < a.D ? lane0 : 0;
                    own[c].load(src + at * ES);
                    up[c].load(grad + at * ES);
                    if constexpr (PAR == kParLoad)
                        if (kt[c].in) par[c].load(grad + (int32_t)(at + kt[c].to_partner) * ES);
                }
                return r;
            };
            NormRow next = load(r0);
            for (uint32_t it = r0; it < rows; it += a.rows_per_block) {
                const NormRow r = next;
                gchar* dst = yd + (r.b * a.y[kind].sb + r.s * a.y[kind].ss + r.n * a.y[kind].sn) * ES;
                const float* cosv = norm_lds + r.k * a.turn.pairs;
                const float* sinv = cosv + a.lds_floats;
                float x[C][8], g[C][8], ss = 0.0f, dot = 0.0f;
#pragma unroll
                for (int c = 0; c < C; ++c) up[c].widen(g[c]);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    own[c].widen(x[c]);
                    if (!kt[c].in) continue;
                    ChunkTurn back = kt[c];        // turned back: the other sign
                    back.first = !back.first;
                    if constexpr (PAR != kParNear) {
                        float p[8];
                        if constexpr (PAR == kParOwn) up[C - 1 - c].widen(p);
                        else par[c].widen(p);
                        turn_chunk(g[c], p, back, false, cosv, sinv);
                    } else {
                        turn_back_adjacent(g[c], kt[c], cosv, sinv);
                    }
                }
                next = load(it + a.rows_per_block);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const bool in = (c * a.T + tt) * 8 < a.D;
                    float s = 0.0f, d = 0.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        s = __builtin_fmaf(x[c][e], x[c][e], s);
                        d = __builtin_fmaf(g[c][e] * w[c][e], x[c][e], d);
                    }
                    ss += in ? s : 0.0f;
                    dot += in ? d : 0.0f;
                }
                const float inv = rsqrtf(__builtin_fmaf(lanes_sum(ss, a.T), a.inv_d, a.eps));
                const float m = lanes_sum(dot, a.T) * inv * a.inv_d;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const uint32_t lane0 = (c * a.T + tt) * 8;
                    float d[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float n = x[c][e] * inv;
                        dw[kind][c][e] = __builtin_fmaf(g[c][e], n, dw[kind][c][e]);
                        d[e] = inv * (g[c][e] * w[c][e] - n * m);
                    }
                    if (lane0 < a.D) store_chunk<DT>(dst + lane0 * ES, d);
                }
            }
        }
    }
    if (a.part == nullptr) return;
    // lanes of a wave that hold the same chunk, then the waves
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
#pragma unroll
        for (int c = 0; c < C; ++c) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float v = dw[kind][c][e];
                for (uint32_t d = a.T; d < 64; d <<= 1) v += __shfl_xor(v, (int)d);
                if ((t & 63) < a.T) norm_lds[((t >> 6) * a.T + tt) * 8 + e] = v;
            }
            __syncthreads();
            for (uint32_t j = t; j < a.T * 8; j += kNormThreads) {
                float sum = 0.0f;
                for (int w = 0; w < kNormWaves; ++w) sum += norm_lds[w * a.T * 8 + j];
                const uint32_t lane = c * a.T * 8 + j;
                if (lane < a.D) a.part[((uint64_t)blockIdx.x * 2 + kind) * a.D + lane] = sum;
            }
        }
}

// The weights' gradients: the blocks' sums added in a fixed order, rounded
// once. A block takes 4 lanes of one weight, a thread a strand of partial sums:
// many small blocks, since each sum has to come from another chiplet's cache.
// (16 lanes a block, 64 strands: 7.6 us for 1024 sums of 128 lanes; 256 strands
// of 16 lanes 9.2.)
struct NormWeightArgs {
    const float* part;
    void* dw[2];
    uint32_t blocks, D;
    int32_t wdt;
};

constexpr int kStrands = 256;

__global__ void __launch_bounds__(kStrands) rope_norm_weight_grad_kernel(NormWeightArgs a)
{
    __shared__ float sums[kStrands / 64][4];
    const uint32_t strand = threadIdx.x, j = blockIdx.x * 4;
    const int kind = blockIdx.y;
    if (a.dw[kind] == nullptr) return;
    float sum[4] = {};
#pragma unroll 4
    for (uint32_t b = strand; b < a.blocks; b += kStrands) {
        const float* p = a.part + ((uint64_t)b * 2 + kind) * a.D + j;
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += j + e < a.D ? p[e] : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        sum[e] = lanes_sum(sum[e], 64);
        if ((strand & 63) == 0) sums[strand >> 6][e] = sum[e];
    }
    __syncthreads();
    const uint32_t at = j + strand;
    if (strand >= 4 || at >= a.D) return;
    const float v = (sums[0][strand] + sums[1][strand]) + (sums[2][strand] + sums[3][strand]);
    switch (a.wdt) {
    case ROPE_DTYPE_F32: Store<ROPE_DTYPE_F32>::store1(a.dw[kind], at, v); break;
    case ROPE_DTYPE_F16: Store<ROPE_DTYPE_F16>::store1(a.dw[kind], at, v); break;
    default: Store<ROPE_DTYPE_BF16>::store1(a.dw[kind], at, v); break;
    }
}

}  // namespace
}  // namespace rope
