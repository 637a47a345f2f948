// rope_lora_kernels.hpp -- a head projection with each token's own low-rank
// adapter, and a rotary epilogue: y = rotate(x . w^T + h . b_i^T) with
// h = s_i (x . a_i^T), i the token's adapter.
// Included by rope_lora.hip, next to the host code that launches them.
//
// Two launches. The first computes h, M x R fp32 numbers in the workspace:
// a token reads its own adapter's R rows of a. The second is the projection,
// which adds h . b_i^T to its fp32 accumulators before it rotates them, so
// that neither the shared product nor the adapters' makes a round trip
// through memory.
#pragma once

#include "rope_proj_kernels.hpp"

namespace rope {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

struct LoraArgs {
    const uint16_t* a;     // (count, R, K)
    const uint16_t* b;     // (count, N, R)
    const int32_t* ids;    // (M); outside [0, count): none
    const float* scales;   // (count) or NULL
    float* h;              // (M, R) workspace
    int32_t count, R;
};

struct LoraProjArgs : ProjArgs {
    LoraArgs l;
};

// The token's adapter, or -1.
__device__ __forceinline__ int32_t lora_id(const LoraArgs& l, int32_t m)
{
    const int32_t i = l.ids[m];
    return i >= 0 && i < l.count ? i : -1;
}

// 8 16-bit values as fp32.
template <int DT>
__device__ __forceinline__ void widen8(const v4u& q, float (&f)[8])
{
    Lanes<DT> t;
    t.unpack(q);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = t.v[k];
}

// ---------------------------------------------------------------------------
// h by dot products: a wave per (token, rank), 16 bytes of x and of a per lane
// and step, the 64 partial sums joined by shuffles in a fixed order. For few
// tokens it is bound by the latency of one pass over a row; each of R/4
// blocks of a token reads x again, from L2.
// ---------------------------------------------------------------------------
constexpr int kShrinkWaves = 4;

template <int DT>
__global__ void __launch_bounds__(64 * kShrinkWaves) rope_lora_shrink_kernel(LoraArgs l, const uint16_t* x, int32_t M,
                                                                            int32_t K)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = blockIdx.y * kShrinkWaves + wave;
    if (r >= l.R) return;
    for (int32_t m = blockIdx.x; m < M; m += gridDim.x) {
        const int32_t id = lora_id(l, m);
        if (id < 0) continue;
        const uint16_t* xr = x + (int64_t)m * K;
        const uint16_t* ar = l.a + ((int64_t)id * l.R + r) * K;
        float sum = 0.0f;
        for (int32_t k = lane * 8; k < K; k += 512) {
            float fx[8], fa[8];
            widen8<DT>(*reinterpret_cast<const v4u*>(xr + k), fx);
            widen8<DT>(*reinterpret_cast<const v4u*>(ar + k), fa);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(fx[e], fa[e], sum);
        }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
        if (lane == 0) l.h[(int64_t)m * l.R + r] = l.scales != nullptr ? sum * l.scales[id] : sum;
    }
}

template <int DT>
__device__ __forceinline__ f32x4 mfma16(const v4u& a, const v4u& b, const f32x4& c)
{
    if constexpr (DT == ROPE_DTYPE_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
}

// ---------------------------------------------------------------------------
// The adapters' part of the tiled projections: after the K loop, R more k for
// each adapter of the wave's tokens, on the same accumulators. A fragment of
// 32 tokens that share an adapter (a prompt's) goes straight into them; one
// of several adapters takes each in turn into cleared accumulators and adds
// only its own tokens' values (not a product with h = 0, which an infinity
// or NaN in one adapter would carry into every other's tokens).
// h is fp32 and the MFMA takes 16 bits: h = p0 + p1 (+ p2) in bf16, each the
// rest of the one before it rounded to 8 bits, two parts for 16-bit outputs
// (what is left is below 2^-16 of h, the output rounds at 2^-9 or 2^-12) and
// three for fp32 (2^-24). fp16 weights take the same route, b = q0 + q1
// exactly (11 bits in two of 8): h may exceed fp16's range.
// ---------------------------------------------------------------------------

// v rounded to bf16, as 8 lanes; v becomes what is left.
__device__ __forceinline__ v4u take_bf16(float (&v)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        w[k] = Store<ROPE_DTYPE_BF16>::narrow(f32x2{v[2 * k], v[2 * k + 1]});
        const f32x2 f = Store<ROPE_DTYPE_BF16>::widen(w[k]);
        v[2 * k] -= f.x;
        v[2 * k + 1] -= f.y;
    }
    return v4u{w[0], w[1], w[2], w[3]};
}

// One 32 x 32 tile: c += (8 k of b per lane, BQ parts) x (of h, `parts`).
// COLS: tokens are the tile's columns (square tiles), else its rows.
template <int BQ, bool COLS>
__device__ __forceinline__ void lora_mfma(f32x16& c, const v4u (&b)[BQ], const v4u (&h)[3], int parts)
{
#pragma unroll
    for (int p = 0; p < 3; ++p)
        if (p < 2 || parts > 2)
#pragma unroll
            for (int q = 0; q < BQ; ++q)
                c = COLS ? proj_mfma<ROPE_DTYPE_BF16>(b[q], h[p], c) : proj_mfma<ROPE_DTYPE_BF16>(h[p], b[q], c);
}

// The tiles of 32 tokens (this lane's id and row of h) and NT x 32 output
// lanes from n0, at(nt) their accumulators.
template <int DT, int NT, bool COLS, class AT>
__device__ __forceinline__ void lora_add_tiles(const LoraProjArgs& a, int32_t m, int32_t n0, int lane, AT at)
{
    constexpr int BQ = DT == ROPE_DTYPE_F16 ? 2 : 1;
    const LoraArgs& l = a.l;
    const int parts = a.ydt == ROPE_DTYPE_F32 ? 3 : 2;
    if (l.count == 0) return;                             // no adapters: nothing in l may be read
    // tokens past the last repeat it (their results are never stored)
    m = min(m, a.M - 1);
    const int32_t id = lora_id(l, m);
    const int rl = (lane >> 5) * 8;                       // the lane's 8 of each 16 ranks
    uint64_t todo = __ballot(id >= 0);
    while (todo != 0) {
        const int32_t cur = __builtin_amdgcn_readlane(id, (int)__builtin_ctzll(todo));
        const bool mine = id == cur;
        const uint64_t same = __ballot(mine);
        const bool all = same == ~0ull;
        f32x16 d[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) d[nt] = all ? at(nt) : f32x16{};
        for (int r = 0; r < l.R; r += 16) {
            const bool live = r + rl < l.R;               // R may end halfway through a step
            float hv[8] = {};
            if (live && mine) {
                const float4* hp = reinterpret_cast<const float4*>(l.h + (int64_t)m * l.R + r + rl);
                const float4 h0 = hp[0], h1 = hp[1];
                hv[0] = h0.x; hv[1] = h0.y; hv[2] = h0.z; hv[3] = h0.w;
                hv[4] = h1.x; hv[5] = h1.y; hv[6] = h1.z; hv[7] = h1.w;
            }
            v4u hp[3];
            hp[0] = take_bf16(hv);
            hp[1] = take_bf16(hv);
            hp[2] = take_bf16(hv);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int32_t n = min(n0 + nt * 32 + (lane & 31), a.N - 1);
                v4u b[BQ] = {};
                if (live) b[0] = *reinterpret_cast<const v4u*>(l.b + ((int64_t)cur * a.N + n) * l.R + r + rl);
                if constexpr (DT == ROPE_DTYPE_F16) {
                    float bv[8];
                    widen8<DT>(b[0], bv);
                    b[0] = take_bf16(bv);
                    b[1] = take_bf16(bv);
                }
                lora_mfma<BQ, COLS>(d[nt], b, hp, parts);
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (all) {
                at(nt) = d[nt];
            } else {
                // accumulator register e of lane i: column i%32, row 8*(e/4) + 4*(i/32) + e%4
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const bool own = COLS ? mine
                                          : ((same >> (8 * (e >> 2) + 4 * (lane >> 5) + (e & 3))) & 1u) != 0;
                    at(nt)[e] = own ? at(nt)[e] + d[nt][e] : at(nt)[e];
                }
            }
        }
        todo &= ~same;
    }
}

template <>
struct ProjAdapters<LoraProjArgs> {
    static constexpr bool kAny = true;

    // square tiles: the wave's 4 x 4 tiles, [nt][mt], tokens in columns
    template <int DT>
    __device__ static __forceinline__ void add_square(const LoraProjArgs& a, f32x16 (&acc)[4][4], int32_t m0,
                                                      int32_t n0, int lane)
    {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
            lora_add_tiles<DT, 4, true>(a, m0 + mt * 32 + (lane & 31), n0, lane,
                                        [&](int nt) -> f32x16& { return acc[nt][mt]; });
    }

    // tiles of whole heads: [mt][nt], tokens in rows
    template <int DT, int MT, int NT>
    __device__ static __forceinline__ void add_heads(const LoraProjArgs& a, f32x16 (&acc)[MT][NT], int32_t m0,
                                                     int32_t n0, int lane)
    {
        // one tile at a time: cleared accumulators for all NT beside the
        // wave's own would not fit its 168 registers
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                lora_add_tiles<DT, 1, false>(a, m0 + mt * 32 + (lane & 31), n0 + nt * 32, lane,
                                             [&](int) -> f32x16& { return acc[mt][nt]; });
    }
};

// One table value of runtime type.
__device__ __forceinline__ float table_value(const void* t, int tdt, int64_t i)
{
    switch (tdt) {
    case ROPE_DTYPE_F32: return Store<ROPE_DTYPE_F32>::load1(t, i);
    case ROPE_DTYPE_F16: return Store<ROPE_DTYPE_F16>::load1(t, i);
    default: return Store<ROPE_DTYPE_BF16>::load1(t, i);
    }
}

// sum_r h[m,r] b[id,n,r] in fp32, r ascending.
template <int DT>
__device__ __forceinline__ float lora_dot(const LoraArgs& l, const float* h, int32_t id, int64_t n, int64_t N)
{
    const uint16_t* br = l.b + ((int64_t)id * N + n) * l.R;
    float sum = 0.0f;
    for (int r = 0; r < l.R; r += 8) {
        float fb[8];
        widen8<DT>(*reinterpret_cast<const v4u*>(br + r), fb);
        const float4 h0 = *reinterpret_cast<const float4*>(h + r), h1 = *reinterpret_cast<const float4*>(h + r + 4);
        sum = __builtin_fmaf(h0.x, fb[0], sum);
        sum = __builtin_fmaf(h0.y, fb[1], sum);
        sum = __builtin_fmaf(h0.z, fb[2], sum);
        sum = __builtin_fmaf(h0.w, fb[3], sum);
        sum = __builtin_fmaf(h1.x, fb[4], sum);
        sum = __builtin_fmaf(h1.y, fb[5], sum);
        sum = __builtin_fmaf(h1.z, fb[6], sum);
        sum = __builtin_fmaf(h1.w, fb[7], sum);
    }
    return sum;
}

// ---------------------------------------------------------------------------
// General projection: any head of up to 1024 lanes, any slice. A block takes
// 16 tokens and one head; its waves take the head's 16-lane fragments in
// turn, four at a time, with 16x16x32 MFMAs whose operands come straight from
// memory (a lane holds 8 consecutive k of one row of w or of x). The head's
// fp32 values meet in LDS, where the adapters' part is added and partners are
// found whatever the slice.
// ---------------------------------------------------------------------------
constexpr int kHeadTokens = 16;
constexpr int kHeadPitch = ROPE_D_LIMIT + 4;

template <int DT>
__global__ void __launch_bounds__(256) rope_lora_head_kernel(LoraProjArgs g, int tdt, int heads)
{
    __shared__ __attribute__((aligned(16))) float P[kHeadTokens * kHeadPitch];
    const ProjArgs& a = g;
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int fr = lane & 15, fk = (lane >> 4) * 8;
    const int nf = a.Dh / 16;
    const int64_t tiles = (int64_t)((a.M + kHeadTokens - 1) / kHeadTokens) * heads;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int32_t hd = (int32_t)(tile % heads);
        const int32_t m0 = (int32_t)(tile / heads) * kHeadTokens;
        const int64_t n0 = (int64_t)hd * a.Dh;
        const uint16_t* xr = a.x + (int64_t)min(m0 + fr, a.M - 1) * a.K + fk;
        for (int f0 = wave * 4; f0 < nf; f0 += 16) {
            f32x4 acc[4] = {};
            const uint16_t* wr[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) wr[j] = a.w + (n0 + min(f0 + j, nf - 1) * 16 + fr) * a.K + fk;
            for (int32_t k = 0; k < a.K; k += 32) {
                const v4u xv = *reinterpret_cast<const v4u*>(xr + k);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[j] = mfma16<DT>(*reinterpret_cast<const v4u*>(wr[j] + k), xv, acc[j]);
            }
            // accumulator register e of lane l: output lane 4*(l/16) + e, token l%16
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (f0 + j < nf)
                    *reinterpret_cast<f32x4*>(&P[fr * kHeadPitch + (f0 + j) * 16 + (lane >> 4) * 4]) = acc[j];
        }
        __syncthreads();
        if (g.l.count > 0) {
            for (int i = threadIdx.x; i < kHeadTokens * a.Dh; i += 256) {
                const int t = i / a.Dh, j = i - t * a.Dh;
                if (m0 + t >= a.M) continue;
                const int32_t id = lora_id(g.l, m0 + t);
                if (id >= 0)
                    P[t * kHeadPitch + j] += lora_dot<DT>(g.l, g.l.h + (int64_t)(m0 + t) * g.l.R, id, n0 + j, a.N);
            }
            __syncthreads();
        }
        for (int i = threadIdx.x; i < kHeadTokens * a.Dh; i += 256) {
            const int t = i / a.Dh, j = i - t * a.Dh;
            const int32_t m = m0 + t;
            if (m >= a.M) continue;
            float v = P[t * kHeadPitch + j];
            const int rel = j - a.start;
            if (rel >= 0 && rel < a.L) {
                const bool first = rel % (2 * a.half) < a.half;
                const float xp = P[t * kHeadPitch + j + (first ? a.half : -a.half)];
                const int32_t b = (int32_t)fast_div((uint32_t)m, a.s_div), s = m - b * a.S;
                const float c = table_value(a.r1, tdt, b * a.t1b + s * a.t1s + hd * a.t1n + rel);
                const float sn = table_value(a.r2, tdt, b * a.t2b + s * a.t2s + hd * a.t2n + rel);
                v = rotate_own<false>(v, xp, c, sn, first);
            }
            const int64_t yo = (int64_t)m * a.N + n0 + j;
            if (a.ydt == ROPE_DTYPE_F32) Store<ROPE_DTYPE_F32>::store1(a.y, yo, v);
            else Store<DT>::store1(a.y, yo, v);
        }
        __syncthreads();      // the next tile overwrites P
    }
}

}  // namespace
}  // namespace rope
