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

// h[m,r] of the token's adapter by the whole wave: 16 bytes of x and of a per
// lane and step, the 64 partial sums joined by shuffles in a fixed order.
template <int DT>
__device__ __forceinline__ void lora_dot_k(const LoraArgs& l, const uint16_t* x, int32_t m, int32_t id, int r,
                                           int32_t K, int lane)
{
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

// ---------------------------------------------------------------------------
// h by dot products, a wave per (token, rank): for few tokens. Bound by the
// latency of one pass over a row; each of a token's R/4 blocks reads x again,
// from L2.
// ---------------------------------------------------------------------------
constexpr int kShrinkWaves = 4;

template <int DT>
__global__ void __launch_bounds__(64 * kShrinkWaves) rope_lora_shrink_kernel(LoraArgs l, const uint16_t* x, int32_t K)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = blockIdx.y * kShrinkWaves + wave;
    if (r >= l.R) return;
    const int32_t m = (int32_t)blockIdx.x;
    const int32_t id = lora_id(l, m);
    if (id >= 0) lora_dot_k<DT>(l, x, m, id, r, K, lane);
}

// ---------------------------------------------------------------------------
// h by MFMA, for prompts: a block takes 32 tokens and 32 ranks, its waves a
// quarter of K each (whole 64-k blocks, one 128-byte line of each row), with
// 32x32x16 MFMAs whose operands come straight from memory; the four partial
// tiles meet in LDS in a fixed order. The k of a 64-k block may go to any MFMA
// slot as long as a and x agree: lane l takes 16 bytes (8 k) at (2j + l/32) *
// 16 of its row's line in step j, so a step's 64 loads fill half lines that
// the next steps complete. Tokens of several adapters take one pass over K
// for each; a block with more than kShrinkPasses of them takes its tokens
// one by one with dot products, as the kernel above does: a pass costs the
// block about what 8 tokens' dot products do.
// ---------------------------------------------------------------------------
constexpr int kShrinkPasses = 4;

template <int DT>
__global__ void __launch_bounds__(256) rope_lora_shrink_tile_kernel(LoraArgs l, const uint16_t* x, int32_t M, int32_t K)
{
    __shared__ float part[4][32][33];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int fr = lane & 31, hw = lane >> 5;
    const int32_t m0 = (int32_t)blockIdx.x * 32;
    const int r0 = (int)blockIdx.y * 32;
    const int32_t m = min(m0 + fr, M - 1);
    const int32_t id = lora_id(l, m);
    uint64_t todo = __ballot(id >= 0);
    int passes = 0;
    for (uint64_t t = todo; t != 0; ++passes)
        t &= ~__ballot(id == __builtin_amdgcn_readlane(id, (int)__builtin_ctzll(t)));
    if (passes > kShrinkPasses) {
        // the same for every wave: all read the same ids
        for (int i = wave; i < 32 * 32; i += 4) {
            const int t = i >> 5, r = r0 + (i & 31);
            if (m0 + t >= M || r >= l.R) continue;
            const int32_t own = __builtin_amdgcn_readlane(id, t);
            if (own < 0) continue;
            lora_dot_k<DT>(l, x, m0 + t, own, r, K, lane);
        }
        return;
    }
    const int32_t blocks = K / 64;
    const uint16_t* xr = x + (int64_t)m * K + hw * 8;
    while (todo != 0) {
        const int32_t cur = __builtin_amdgcn_readlane(id, (int)__builtin_ctzll(todo));
        const uint16_t* ar = l.a + ((int64_t)cur * l.R + min(r0 + fr, l.R - 1)) * K + hw * 8;
        f32x16 acc = {};
#pragma unroll 2
        for (int32_t kb = wave; kb < blocks; kb += 4) {
            v4u fx[4], fa[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                fx[j] = *reinterpret_cast<const v4u*>(xr + (int64_t)kb * 64 + j * 16);
                fa[j] = *reinterpret_cast<const v4u*>(ar + (int64_t)kb * 64 + j * 16);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) acc = proj_mfma<DT>(fa[j], fx[j], acc);
        }
        // register e of lane i: rank 8*(e/4) + 4*(i/32) + e%4, token i%32
#pragma unroll
        for (int e = 0; e < 16; ++e) part[wave][fr][8 * (e >> 2) + 4 * hw + (e & 3)] = acc[e];
        __syncthreads();
        const float s = l.scales != nullptr ? l.scales[cur] : 1.0f;
        for (int i = threadIdx.x; i < 32 * 32; i += 256) {
            const int t = i >> 5, r = i & 31;
            // the token's adapter from the lane that holds it: every lane of
            // a wave reads it, so before any branch
            const int32_t own = __shfl(id, t);
            const float sum = (part[0][t][r] + part[1][t][r]) + (part[2][t][r] + part[3][t][r]);
            if (own == cur && m0 + t < M && r0 + r < l.R) l.h[(int64_t)(m0 + t) * l.R + r0 + r] = sum * s;
        }
        todo &= ~__ballot(id == cur);
        if (todo != 0) __syncthreads();      // the next pass rewrites part
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
// lanes from n0, at(nt) their accumulators; nothing unless `any`.
template <int DT, int NT, bool COLS, class AT>
__device__ __forceinline__ void lora_add_tiles(const LoraProjArgs& a, int32_t m, int32_t n0, int lane, bool any,
                                               AT at)
{
    constexpr int BQ = DT == ROPE_DTYPE_F16 ? 2 : 1;
    const LoraArgs& l = a.l;
    const int parts = a.ydt == ROPE_DTYPE_F32 ? 3 : 2;
    // tokens past the last repeat it (their results are never stored)
    m = min(m, a.M - 1);
    const int32_t id = any ? lora_id(l, m) : -1;
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

    // One step of 16 ranks of a square tile's wave whose 128 tokens share an
    // adapter: b of its 4 x 32 output lanes and h of its 4 x 32 tokens.
    struct Step {
        v4u b[4];
        float4 h[4][2];
    };
    // A square tile's wave: the adapter that all its tokens have (-1: none
    // has one; kMixed: several) and the first step, fetched while the last K
    // stage's MFMAs run, which hide its latency.
    static constexpr int32_t kMixed = -2;
    struct Square {
        int32_t id;
        Step step;
    };

    template <int DT>
    __device__ static __forceinline__ void find_square(const LoraProjArgs& a, Square& q, int32_t m0, int lane)
    {
        q.id = -1;
        if (a.l.count == 0) return;
        int32_t id[4];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) id[mt] = lora_id(a.l, min(m0 + mt * 32 + (lane & 31), a.M - 1));
        const int32_t first = __builtin_amdgcn_readfirstlane(id[0]);
        const bool same = id[0] == first && id[1] == first && id[2] == first && id[3] == first;
        q.id = __ballot(same) == ~0ull ? first : kMixed;
    }

    __device__ static __forceinline__ void load_step(const LoraProjArgs& a, Step& t, int32_t id, int32_t m0, int32_t n0,
                                                     int r, int lane)
    {
        const LoraArgs& l = a.l;
        // ranks past R (the upper half of a last half step) re-read the lower
        // half; add_step clears h there, and b is finite or its own tokens'
        const int rk = r + (lane >> 5) * 8 < l.R ? r + (lane >> 5) * 8 : r;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
            const int32_t n = min(n0 + nt * 32 + (lane & 31), a.N - 1);
            t.b[nt] = *reinterpret_cast<const v4u*>(l.b + ((int64_t)id * a.N + n) * l.R + rk);
        }
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            const int32_t m = min(m0 + mt * 32 + (lane & 31), a.M - 1);
            const float4* hp = reinterpret_cast<const float4*>(l.h + (int64_t)m * l.R + rk);
            t.h[mt][0] = hp[0];
            t.h[mt][1] = hp[1];
        }
    }

    template <int DT>
    __device__ static __forceinline__ void fetch_square(const LoraProjArgs& a, Square& q, int32_t m0, int32_t n0,
                                                        int lane)
    {
        if (q.id >= 0) load_step(a, q.step, q.id, m0, n0, 0, lane);
    }

    // The products of one step. Its operands are rounded to bf16 parts first;
    // their registers then take the step at `next` (if next < R), whose
    // latency the MFMAs hide.
    template <int DT>
    __device__ static __forceinline__ void add_step(const LoraProjArgs& a, Square& s, f32x16 (&acc)[4][4], int32_t m0,
                                                    int32_t n0, int r, int lane)
    {
        constexpr int BQ = DT == ROPE_DTYPE_F16 ? 2 : 1;
        const bool live = r + (lane >> 5) * 8 < a.l.R;
        v4u b[4][BQ], h[3][4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
            b[nt][0] = live ? s.step.b[nt] : v4u{};
            if constexpr (DT == ROPE_DTYPE_F16) {
                float bv[8];
                widen8<DT>(b[nt][0], bv);
                b[nt][0] = take_bf16(bv);
                b[nt][1] = take_bf16(bv);
            }
        }
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            const float4 h0 = s.step.h[mt][0], h1 = s.step.h[mt][1];
            float v[8] = {h0.x, h0.y, h0.z, h0.w, h1.x, h1.y, h1.z, h1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = live ? v[e] : 0.0f;
#pragma unroll
            for (int p = 0; p < 3; ++p) h[p][mt] = take_bf16(v);
        }
        if (r + 16 < a.l.R) load_step(a, s.step, s.id, m0, n0, r + 16, lane);
        // one part of h at a time over all 16 tiles: MFMAs on one
        // accumulator are 16 apart
        auto part = [&](const v4u (&hp)[4]) {
#pragma unroll
            for (int q = 0; q < BQ; ++q)
#pragma unroll
                for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt)
                        acc[nt][mt] = proj_mfma<ROPE_DTYPE_BF16>(b[nt][q], hp[mt], acc[nt][mt]);
        };
        part(h[0]);
        part(h[1]);
        if (a.ydt == ROPE_DTYPE_F32) part(h[2]);
    }

    // square tiles: the wave's 4 x 4 tiles, [nt][mt], tokens in columns
    template <int DT>
    __device__ static __forceinline__ void add_square(const LoraProjArgs& a, Square& q, f32x16 (&acc)[4][4],
                                                      int32_t m0, int32_t n0, int lane)
    {
        // one loop behind the other, each with no turns where it does not
        // apply: branches that the 256 accumulators meet behind make the
        // compiler spill them
        const int fast = q.id >= 0 ? a.l.R : 0;
#pragma unroll 1
        for (int r = 0; r < fast; r += 16) add_step<DT>(a, q, acc, m0, n0, r, lane);
        const bool mixed = q.id == kMixed;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
            lora_add_tiles<DT, 4, true>(a, m0 + mt * 32 + (lane & 31), n0, lane, mixed,
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
                lora_add_tiles<DT, 1, false>(a, m0 + mt * 32 + (lane & 31), n0 + nt * 32, lane, a.l.count > 0,
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
// Few tokens: bound by reading w once. A block takes a unit of 32 output lanes
// (two 16-lane fragments) and up to 64 tokens; its W waves take 64-k blocks of
// K in turn (one 128-byte line of each row of w), with 16x16x32 MFMAs whose
// operands come straight from memory: w is read by one wave only, and x, which
// every block reads, comes from L2. The waves' partial tiles meet in LDS in a
// fixed order; then a thread holds one token and 4 lanes of both fragments,
// adds the adapter's part by dot products (each token has its own b: MFMA
// tiles would be one token wide) and rotates.
// Where partners lie whole fragments apart, a unit is a fragment of a group's
// first half and the matching one of its second, so that partners meet in one
// thread; otherwise fragments go in order.
// ---------------------------------------------------------------------------
struct FewArgs : LoraProjArgs {
    int32_t apart;           // partners are whole fragments apart
    int32_t head_units;      // units of a head: Dh / 32
    int32_t slice_units;     // apart: units of a head's slice, its first ones
    int32_t first_frag, slice_frags, half_frags;   // apart: of the slice, in 16 lanes
};

// The unit's two fragments, as first lanes within the head; *turned: both in
// the slice, the second holding the first's partners.
__device__ __forceinline__ void few_unit(const FewArgs& a, int32_t u, int32_t (&lane0)[2], bool* turned)
{
    *turned = a.apart && u < a.slice_units;
    if (*turned) {
        const int32_t g = u / a.half_frags, k = u - g * a.half_frags;
        lane0[0] = (a.first_frag + g * 2 * a.half_frags + k) * 16;
        lane0[1] = lane0[0] + a.half_frags * 16;
        return;
    }
    // the fragments outside the slice (apart), or all of them, in order
#pragma unroll
    for (int f = 0; f < 2; ++f) {
        const int32_t j = 2 * (u - a.slice_units) + f;
        lane0[f] = (j < a.first_frag ? j : j + a.slice_frags) * 16;
    }
}

template <int DT, int MT, int W>
__global__ void __launch_bounds__(64 * W) rope_lora_few_kernel(FewArgs a, int tdt)
{
    __shared__ f32x4 part[W][2][MT][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, quad = lane >> 4;
    const int32_t hd = (int32_t)blockIdx.x / a.head_units;
    int32_t lane0[2];
    bool turned;
    few_unit(a, (int32_t)blockIdx.x - hd * a.head_units, lane0, &turned);
    const int64_t n0 = (int64_t)hd * a.Dh;
    const int32_t m0 = (int32_t)blockIdx.y * (16 * MT);

    const uint16_t* wr[2];
    const uint16_t* xr[MT];
#pragma unroll
    for (int f = 0; f < 2; ++f) wr[f] = a.w + (n0 + lane0[f] + fr) * a.K + quad * 8;
#pragma unroll
    for (int t = 0; t < MT; ++t) xr[t] = a.x + (int64_t)min(m0 + t * 16 + fr, a.M - 1) * a.K + quad * 8;
    f32x4 acc[2][MT] = {};
    const int32_t blocks = a.K / 64;
#pragma unroll 2
    for (int32_t kb = wave; kb < blocks; kb += W) {
        v4u fw[2][2], fx[MT][2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int f = 0; f < 2; ++f)
                fw[f][s] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(wr[f] + kb * 64 + s * 32));
#pragma unroll
            for (int t = 0; t < MT; ++t) fx[t][s] = *reinterpret_cast<const v4u*>(xr[t] + kb * 64 + s * 32);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int t = 0; t < MT; ++t) acc[f][t] = mfma16<DT>(fw[f][s], fx[t][s], acc[f][t]);
    }
    // register e of lane i: output lane 4*(i/16) + e of the fragment, token i%16
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int t = 0; t < MT; ++t) part[wave][f][t][lane] = acc[f][t];
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * MT; i += 64 * W) {
        const int t = i >> 6;
        const int32_t m = m0 + t * 16 + (i & 15);
        if (m >= a.M) continue;
        float v[2][4];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            f32x4 sum = part[0][f][t][i & 63];
#pragma unroll
            for (int w = 1; w < W; ++w) sum += part[w][f][t][i & 63];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[f][e] = sum[e];
        }
        const int q4 = ((i & 63) >> 4) * 4;        // first of the thread's 4 lanes in each fragment
        const int32_t id = a.l.count > 0 ? lora_id(a.l, m) : -1;
        if (id >= 0) {
            const float* h = a.l.h + (int64_t)m * a.l.R;
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[f][e] += lora_dot<DT>(a.l, h, id, n0 + lane0[f] + q4 + e, a.N);
        }
        if (a.L > 0) {
            const int32_t b = (int32_t)fast_div((uint32_t)m, a.s_div), s = m - b * a.S;
            const int64_t o1 = b * a.t1b + s * a.t1s + hd * a.t1n, o2 = b * a.t2b + s * a.t2s + hd * a.t2n;
            if (turned) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int32_t r = lane0[0] + q4 + e - a.start, rp = r + a.half;
                    const float x0 = v[0][e], x1 = v[1][e];
                    v[0][e] = rotate_own<false>(x0, x1, table_value(a.r1, tdt, o1 + r), table_value(a.r2, tdt, o2 + r), true);
                    v[1][e] = rotate_own<false>(x1, x0, table_value(a.r1, tdt, o1 + rp), table_value(a.r2, tdt, o2 + rp), false);
                }
            } else if (!a.apart) {
                // adjacent pairs, which a thread's 4 lanes hold whole
#pragma unroll
                for (int f = 0; f < 2; ++f)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const int32_t r = lane0[f] + q4 + e - a.start;
                        if (r < 0 || r >= a.L) continue;
                        const float x0 = v[f][e], x1 = v[f][e + 1];
                        v[f][e] = rotate_own<false>(x0, x1, table_value(a.r1, tdt, o1 + r), table_value(a.r2, tdt, o2 + r), true);
                        v[f][e + 1] = rotate_own<false>(x1, x0, table_value(a.r1, tdt, o1 + r + 1),
                                                        table_value(a.r2, tdt, o2 + r + 1), false);
                    }
            }
        }
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const int64_t yo = (int64_t)m * a.N + n0 + lane0[f] + q4;
            if (a.ydt == ROPE_DTYPE_F32) {
                *reinterpret_cast<float4*>(static_cast<float*>(a.y) + yo) = float4{v[f][0], v[f][1], v[f][2], v[f][3]};
            } else {
                *reinterpret_cast<v2u*>(static_cast<uint16_t*>(a.y) + yo) =
                    v2u{Store<DT>::narrow(f32x2{v[f][0], v[f][1]}), Store<DT>::narrow(f32x2{v[f][2], v[f][3]})};
            }
        }
    }
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
