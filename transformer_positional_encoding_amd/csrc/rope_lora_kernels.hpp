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
    const int32_t* ids;    // (M) adapter of each token; outside [0, count): none
    const float* scales;   // (count) or NULL
    float* h;              // (M, R) workspace
    int32_t count, R;
    // the tiled kernels' rows (see the sort): the token of each, the adapter
    // of every 32, and how many there are
    const int32_t* order;
    const int32_t* group_ids;
    const int32_t* rows;
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
// Rows for the tiled kernels: the tokens in the order of their adapters (those
// without one last), tokens of one adapter in their own order, each adapter's
// rows filled up to whole groups of 32 with gaps (-1). A 32-token column of a
// tile then has one adapter whatever the batch looks like: its products go
// straight into the accumulators, from operands fetched ahead. (With rows
// packed, a column of several took a pass for each into cleared accumulators,
// whose operands came 1.9 us apart under load: 100 us more than this on 8190
// tokens of 8 adapters.) The gaps cost up to 31 rows an adapter.
// A counting sort by one block: its 16 waves count a sixteenth of the tokens
// each, the counts are summed over adapters and waves, and the waves place
// their tokens, a token's rank among its 64 from the ballots of its adapter's
// bits. No order of execution enters the result.
// Lanes of a wave hand counts and places to one another through LDS; the
// hardware keeps a wave's LDS accesses in order, and wave_lds() tells the
// compiler that other lanes' reads and writes lie on either side.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortBins = kLoraSortAdapters + 1;   // and one for none
constexpr int kSortKept = 16;                      // tokens a lane keeps in registers: 16384 tokens in all

__device__ __forceinline__ void wave_lds()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__global__ void __launch_bounds__(kSortThreads) rope_lora_sort_kernel(const int32_t* ids, int32_t count, int32_t M,
                                                                     int32_t* order, int32_t* group_ids, int32_t* rows)
{
    static_assert(kSortBins <= kSortThreads, "a thread for each bin");
    __shared__ int32_t at[kSortWaves][kSortBins];
    __shared__ int32_t sums[kSortWaves];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int bins = count + 1;
    int bits = 1;
    while ((1 << bits) < bins) ++bits;
    for (int w = 0; w < kSortWaves; ++w)
        if (t < bins) at[w][t] = 0;
    __syncthreads();
    const int64_t seg = (((int64_t)M + kSortThreads - 1) / kSortThreads) * 64;    // tokens of a wave, whole 64s
    const int64_t begin = wave * seg, end = min((int64_t)M, begin + seg);
    // (a token past the last repeats it: a branch around each load would wait
    // for them one by one)
    const auto key = [&](int64_t m) {
        const int32_t i = ids[min(m, (int64_t)M - 1)];
        return i >= 0 && i < count ? i : count;
    };
    // the wave's first tokens stay in registers: their loads go out together
    // and serve both walks
    int32_t kept[kSortKept];
#pragma unroll
    for (int i = 0; i < kSortKept; ++i) kept[i] = key(begin + i * 64 + lane);
    // the lanes of 64 tokens that hold this lane's adapter (the whole wave
    // calls it); adding a group's size once spares the LDS 64 additions to one
    // place
    const auto alike = [&](bool live, int32_t k) {
        uint64_t same = __ballot(live);
        for (int i = 0; i < bits; ++i) {
            const uint64_t set = __ballot((k >> i) & 1);
            same &= ((k >> i) & 1) ? set : ~set;
        }
        return same;
    };
    const auto add = [&](int64_t m, int32_t k) {
        const uint64_t same = alike(m < end, k);
        if (m < end && (same & ((1ull << lane) - 1)) == 0) at[wave][k] += __popcll(same);
        wave_lds();
    };
#pragma unroll
    for (int i = 0; i < kSortKept; ++i)
        if (begin + i * 64 < end) add(begin + i * 64 + lane, kept[i]);
    for (int64_t m64 = begin + kSortKept * 64; m64 < end; m64 += 64)
        add(m64 + lane, key(m64 + lane));
    __syncthreads();
    // exclusive sums: over the waves for each bin, then of the bins' padded
    // sizes over the bins
    int32_t total = 0;
    int32_t mine[kSortWaves];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) mine[w] = t < bins ? at[w][t] : 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
        const int32_t n = mine[w];
        mine[w] = total;
        total += n;
    }
    const int32_t padded = (total + 31) & ~31;
    int32_t sum = padded;
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t o = __shfl_up(sum, d);
        if (lane >= d) sum += o;
    }
    if (lane == 63) sums[wave] = sum;
    __syncthreads();
    int32_t before = sum - padded, all = 0;
    for (int w = 0; w < kSortWaves; ++w) {
        if (w < wave) before += sums[w];
        all += sums[w];
    }
    if (t < bins) {
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) at[w][t] = before + mine[w];
        for (int32_t i = total; i < padded; ++i) order[before + i] = -1;
    }
    // gaps to the end of the last tile of either kind
    for (int32_t i = t; i < kLoraTileRows; i += kSortThreads) order[all + i] = -1;
    if (t < kLoraTileRows / 32) group_ids[all / 32 + t] = -1;
    if (t == 0) *rows = all;
    __syncthreads();
    const auto place = [&](int64_t m, int32_t k) {                       // by the whole wave
        const uint64_t same = alike(m < end, k);
        const int32_t to = m < end ? at[wave][k] + __popcll(same & ((1ull << lane) - 1)) : 0;
        wave_lds();
        if (m < end) {
            order[to] = (int32_t)m;
            if ((to & 31) == 0) group_ids[to / 32] = k == count ? -1 : k;
            // the adapter's last token of the 64 moves its place on
            if ((same >> lane) == 1) at[wave][k] = to + 1;
        }
        wave_lds();
    };
#pragma unroll
    for (int i = 0; i < kSortKept; ++i)
        if (begin + i * 64 < end) place(begin + i * 64 + lane, kept[i]);
    for (int64_t m64 = begin + kSortKept * 64; m64 < end; m64 += 64)
        place(m64 + lane, key(m64 + lane));
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
__global__ void __launch_bounds__(64 * kShrinkWaves) rope_lora_shrink_kernel(LoraArgs l, const uint16_t* x, int32_t M,
                                                                            int32_t K)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = blockIdx.y * kShrinkWaves + wave;
    if (r >= l.R) return;
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
        const int32_t id = lora_id(l, (int32_t)m);
        if (id >= 0) lora_dot_k<DT>(l, x, (int32_t)m, id, r, K, lane);
    }
}

// ---------------------------------------------------------------------------
// h by MFMA, for prompts: a block takes 32 sorted rows, whose tokens have one
// adapter, and 32 ranks, its 8 waves an eighth of K each (whole 64-k blocks,
// one 128-byte line of each row), with 32x32x16 MFMAs whose operands come
// straight from memory; the partial tiles meet in LDS in a fixed order. Bound
// by the latency of a wave's few rounds of loads: a prompt of 8190 tokens is
// one block for each compute unit (K 1536, rank 32: 14 us on MI355X, with 4
// waves 19). The k of a 64-k block may go to any MFMA
// slot as long as a and x agree: lane l takes 16 bytes (8 k) at
// (2j + l/32) * 16 of its row's line in step j, so a step's 64 loads fill half
// lines that the next steps complete.
// ---------------------------------------------------------------------------
constexpr int kShrinkTileWaves = 8;

template <int DT>
__global__ void __launch_bounds__(64 * kShrinkTileWaves)
    rope_lora_shrink_tile_kernel(LoraArgs l, const uint16_t* x, int32_t K)
{
    __shared__ float part[kShrinkTileWaves][32][33];
    const int32_t row0 = (int32_t)blockIdx.x * 32;
    if (row0 >= *l.rows) return;
    const int32_t id = l.group_ids[blockIdx.x];
    if (id < 0) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int fr = lane & 31, hw = lane >> 5;
    const int r0 = (int)blockIdx.y * 32;
    const int32_t tok = l.order[row0 + fr];
    const int32_t blocks = K / 64;
    const uint16_t* xr = x + (int64_t)max(tok, 0) * K + hw * 8;
    const uint16_t* ar = l.a + ((int64_t)id * l.R + min(r0 + fr, l.R - 1)) * K + hw * 8;
    f32x16 acc = {};
    for (int32_t kb = wave; kb < blocks; kb += kShrinkTileWaves) {
        v4u fx[4], fa[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            fx[j] = *reinterpret_cast<const v4u*>(xr + (int64_t)kb * 64 + j * 16);
            fa[j] = *reinterpret_cast<const v4u*>(ar + (int64_t)kb * 64 + j * 16);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) acc = proj_mfma<DT>(fa[j], fx[j], acc);
    }
    // register e of lane i: rank 8*(e/4) + 4*(i/32) + e%4, row i%32
#pragma unroll
    for (int e = 0; e < 16; ++e) part[wave][fr][8 * (e >> 2) + 4 * hw + (e & 3)] = acc[e];
    __syncthreads();
    const float s = l.scales != nullptr ? l.scales[id] : 1.0f;
    for (int i = threadIdx.x; i < 32 * 32; i += 64 * kShrinkTileWaves) {
        const int t = i >> 5, r = i & 31;
        const int32_t to = __shfl(tok, t);
        float sum = part[0][t][r];
#pragma unroll
        for (int w = 1; w < kShrinkTileWaves; ++w) sum += part[w][t][r];
        if (to >= 0 && r0 + r < l.R) l.h[(int64_t)to * l.R + r0 + r] = sum * s;
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
// The adapters' part of the tiled projections: after the K loop, R more k on
// the same accumulators, a 32-row column at a time with its own adapter.
// h is fp32 and the MFMA takes 16 bits: h = p0 + p1 (+ p2) in bf16, each the
// rest of the one before it rounded to 8 bits, two parts for 16-bit outputs
// (what is left is below 2^-16 of h, the output rounds at 2^-9 or 2^-12) and
// three for fp32 (2^-24). fp16 weights take the same route, b = q0 + q1
// exactly (11 bits in two of 8): h may exceed fp16's range.
// Columns without an adapter multiply zeros by zeros. A gap's row takes the h
// of token 0; its values are never stored.
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

// 16 bytes of b and 8 of h (fp32) per lane: one step of 16 ranks of 32 rows and
// 32 output lanes.
__device__ __forceinline__ v4u lora_load_b(const LoraProjArgs& a, int32_t id, int32_t n, int r, int lane)
{
    // ranks past R (the upper half of a last half step) re-read the lower half
    const int rk = r + (lane >> 5) * 8 < a.l.R ? r + (lane >> 5) * 8 : r;
    return *reinterpret_cast<const v4u*>(a.l.b + ((int64_t)max(id, 0) * a.N + min(n, a.N - 1)) * a.l.R + rk);
}

struct LoraH {
    float4 q[2];
    __device__ __forceinline__ void load(const LoraProjArgs& a, int32_t tok, int r, int lane)
    {
        const int rk = r + (lane >> 5) * 8 < a.l.R ? r + (lane >> 5) * 8 : r;
        const float4* p = reinterpret_cast<const float4*>(a.l.h + (int64_t)max(tok, 0) * a.l.R + rk);
        q[0] = p[0];
        q[1] = p[1];
    }
};

// The operands of a step, for the MFMAs: zeros unless the lane's ranks exist
// and the column has an adapter.
template <int DT>
__device__ __forceinline__ void lora_parts(const v4u& bl, bool live, v4u (&b)[DT == ROPE_DTYPE_F16 ? 2 : 1])
{
    b[0] = live ? bl : v4u{};
    if constexpr (DT == ROPE_DTYPE_F16) {
        float v[8];
        widen8<DT>(b[0], v);
        b[0] = take_bf16(v);
        b[1] = take_bf16(v);
    }
}

__device__ __forceinline__ void lora_parts(const LoraH& hl, bool live, v4u (&h)[3])
{
    float v[8] = {hl.q[0].x, hl.q[0].y, hl.q[0].z, hl.q[0].w, hl.q[1].x, hl.q[1].y, hl.q[1].z, hl.q[1].w};
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = live ? v[e] : 0.0f;
#pragma unroll
    for (int p = 0; p < 3; ++p) h[p] = take_bf16(v);
}

template <>
struct ProjAdapters<LoraProjArgs> {
    static constexpr bool kAny = true;

    __device__ static __forceinline__ int32_t rows(const LoraProjArgs& a) { return *a.l.rows; }
    __device__ static __forceinline__ int32_t row_token(const LoraProjArgs& a, int32_t row) { return a.l.order[row]; }

    // A square tile's wave: its four columns' adapters and tokens, and the
    // operands of their first step, fetched while the last K stage's MFMAs
    // run, which hide their latency.
    struct Square {
        int32_t id[4];
        int32_t tok[4];
        v4u b[4][4];         // [column][32 output lanes]
        LoraH h[4];
    };

    template <int DT>
    __device__ static __forceinline__ void find_square(const LoraProjArgs& a, Square& q, int32_t m0, int lane)
    {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            q.id[mt] = a.l.group_ids[(m0 >> 5) + mt];
            q.tok[mt] = a.l.order[m0 + mt * 32 + (lane & 31)];
        }
    }

    __device__ static __forceinline__ void load_column(const LoraProjArgs& a, Square& q, int mt, int32_t n0, int r, int lane)
    {
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) q.b[mt][nt] = lora_load_b(a, q.id[mt], n0 + nt * 32 + (lane & 31), r, lane);
        q.h[mt].load(a, q.tok[mt], r, lane);
    }

    template <int DT>
    __device__ static __forceinline__ void fetch_square(const LoraProjArgs& a, Square& q, int32_t n0, int lane)
    {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) load_column(a, q, mt, n0, 0, lane);
    }

    // square tiles: the wave's 4 x 4 tiles, [nt][mt], tokens in columns
    template <int DT>
    __device__ static __forceinline__ void add_square(const LoraProjArgs& a, Square& q, f32x16 (&acc)[4][4], int32_t n0,
                                                      int lane)
    {
        constexpr int BQ = DT == ROPE_DTYPE_F16 ? 2 : 1;
        const bool three = a.ydt == ROPE_DTYPE_F32;
        const bool any = q.id[0] >= 0 || q.id[1] >= 0 || q.id[2] >= 0 || q.id[3] >= 0;
        const int R = any ? a.l.R : 0;
#pragma unroll 1
        for (int r = 0; r < R; r += 16) {
            const bool in = r + (lane >> 5) * 8 < a.l.R;
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                const bool live = in && q.id[mt] >= 0;
                v4u h[3], b[4][BQ];
                lora_parts(q.h[mt], live, h);
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) lora_parts<DT>(q.b[mt][nt], live, b[nt]);
                // the column's next step (past the last: the first again,
                // unused), while the MFMAs of this one and of the other
                // columns run
                load_column(a, q, mt, n0, r + 16 < a.l.R ? r + 16 : 0, lane);
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    if (p == 2 && !three) break;
#pragma unroll
                    for (int k = 0; k < BQ; ++k)
#pragma unroll
                        for (int nt = 0; nt < 4; ++nt)
                            acc[nt][mt] = proj_mfma<ROPE_DTYPE_BF16>(b[nt][k], h[p], acc[nt][mt]);
                }
            }
        }
    }

    // tiles of whole heads: [mt][nt], tokens in rows
    template <int DT, int MT, int NT>
    __device__ static __forceinline__ void add_heads(const LoraProjArgs& a, f32x16 (&acc)[MT][NT], int32_t m0,
                                                     int32_t n0, int lane)
    {
        constexpr int BQ = DT == ROPE_DTYPE_F16 ? 2 : 1;
        const bool three = a.ydt == ROPE_DTYPE_F32;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int32_t id = a.l.group_ids[(m0 >> 5) + mt];
            const int32_t tok = a.l.order[m0 + mt * 32 + (lane & 31)];
            const int R = id >= 0 ? a.l.R : 0;
#pragma unroll 1
            for (int r = 0; r < R; r += 16) {
                const bool live = r + (lane >> 5) * 8 < a.l.R;
                LoraH hl;
                hl.load(a, tok, r, lane);
                v4u bl[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) bl[nt] = lora_load_b(a, id, n0 + nt * 32 + (lane & 31), r, lane);
                v4u h[3];
                lora_parts(hl, live, h);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    v4u b[BQ];
                    lora_parts<DT>(bl[nt], live, b);
#pragma unroll
                    for (int p = 0; p < 3; ++p) {
                        if (p == 2 && !three) break;
#pragma unroll
                        for (int k = 0; k < BQ; ++k) acc[mt][nt] = proj_mfma<ROPE_DTYPE_BF16>(h[p], b[k], acc[mt][nt]);
                    }
                }
            }
        }
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
// Few tokens: bound by reading w once and, from 32 tokens on, by x, which every
// block reads from L2. A block takes a unit of 32 output lanes (two 16-lane
// fragments) and up to 64 tokens; its W waves take 64-k blocks of K in turn
// (one 128-byte line of each row of w), with 16x16x32 MFMAs whose operands
// come straight from memory: w is read by one wave only. The adapters' part
// are dot products (each token has its own b: MFMA tiles would be one token
// wide), dealt to all waves. The waves' tiles and the adapters' part meet in
// LDS in a fixed order; then a thread holds one token and 4 lanes of both
// fragments, and rotates.
// Measured on MI355X (K 1536, 24576 output lanes, rank 16, 64 adapters; with
// the launch of h; us): 1, 16, 32, 64 tokens of an adapter each 24, 31, 38, 54,
// without adapters 20, 23, 28, 38 (w alone: 75 MB, 15 us). The adapters' part
// behind the products, its lines touched before: 25, 31, 41, 60; by the threads
// that store: 26, 33, 37, 53, but in twice the registers. Two units a block
// halve x and read 36 where one reads 40 (64 tokens, no adapters), but 26 for 20
// (1 token) and 65 for 53 (64 adapters: registers).
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

constexpr int kFewWaves = 4;      // 8 are the same within 4% up to 32 tokens, and 50 us for 40 with 64

template <int DT, int MT>
__global__ void __launch_bounds__(64 * kFewWaves) rope_lora_few_kernel(FewArgs a, int tdt)
{
    constexpr int W = kFewWaves;
    __shared__ f32x4 part[W + 1][2][MT][64];     // the waves' tiles, and the adapters' part
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
    // The adapters' part first, so that its loads from all over memory go out
    // at once in all blocks, and the products follow without a wait for them:
    // output lane 4*(i/16) + e of a fragment and token i%16 to lane i, the
    // fragments, e and 16-token tiles dealt to the waves.
    if (a.l.count > 0) {
        constexpr int P = 8 * MT / W;            // of these to a wave
        static_assert(W % MT == 0 && 8 * MT % W == 0, "a wave has one tile of tokens");
        const int t = wave % MT;
        const int32_t m = m0 + t * 16 + fr;
        const int32_t id = m < a.M ? lora_id(a.l, m) : -1;
        float sum[P] = {};
        if (id >= 0) {
            const float* h = a.l.h + (int64_t)m * a.l.R;
            const uint16_t* br[P];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int fe = wave / MT + W / MT * i;
                br[i] = a.l.b + ((int64_t)id * a.N + n0 + lane0[fe / 4] + quad * 4 + fe % 4) * a.l.R;
            }
            for (int r = 0; r < a.l.R; r += 16) {
                const int r8 = r + 8 < a.l.R ? r + 8 : r;      // (of 24 ranks, the last 8 alone)
                v4u bq[P][2];
                float hv[16];
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    bq[i][0] = *reinterpret_cast<const v4u*>(br[i] + r);
                    bq[i][1] = *reinterpret_cast<const v4u*>(br[i] + r8);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 q = *reinterpret_cast<const float4*>(h + (k < 2 ? r : r8) + 4 * (k & 1));
                    hv[4 * k] = q.x;
                    hv[4 * k + 1] = q.y;
                    hv[4 * k + 2] = q.z;
                    hv[4 * k + 3] = q.w;
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (c == 1 && r8 == r) break;
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        float fb[8];
                        widen8<DT>(bq[i][c], fb);
#pragma unroll
                        for (int k = 0; k < 8; ++k) sum[i] = __builtin_fmaf(hv[8 * c + k], fb[k], sum[i]);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int fe = wave / MT + W / MT * i;
            reinterpret_cast<float*>(&part[W][fe / 4][t][lane])[fe % 4] = sum[i];
        }
    }
    f32x4 acc[2][MT] = {};
    const int32_t blocks = a.K / 64;
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
    static_assert(W >= MT, "a thread for each token and four lanes");
    if (threadIdx.x < 64 * MT) {
        const int i = (int)threadIdx.x, t = i >> 6;
        const int32_t m = m0 + t * 16 + (i & 15);
        if (m >= a.M) return;
        float v[2][4];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            f32x4 sum = part[0][f][t][i & 63];
#pragma unroll
            for (int w = 1; w < W; ++w) sum += part[w][f][t][i & 63];
            if (a.l.count > 0) sum += part[W][f][t][i & 63];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[f][e] = sum[e];
        }
        const int q4 = ((i & 63) >> 4) * 4;        // first of the thread's 4 lanes in each fragment
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
