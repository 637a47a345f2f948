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

// The sum over the lanes of a wave that differ in the bits below `width`.
__device__ __forceinline__ float lanes_sum(float v, uint32_t width)
{
    for (uint32_t d = 1; d < width; d <<= 1) v += __shfl_xor(v, (int)d);
    return v;
}

// ---------------------------------------------------------------------------
// General kernels: any dimensions, alignment and slice. A block takes a token,
// its waves the token's rows; cos and sin are evaluated once a token, a row
// stands in LDS for its partners' sake.
// ---------------------------------------------------------------------------
constexpr int kNormThreads = 256;
constexpr int kNormWaves = kNormThreads / 64;
constexpr int kNormLanes = ROPE_D_LIMIT / 64;     // lanes of a row that a thread takes at most

__device__ __forceinline__ void norm_turns(const NormArgs& a, uint32_t tok, float2* cs)
{
    const uint32_t b = fast_div(tok, a.s_div);
    for (uint32_t i = threadIdx.x; i < a.turn.pairs; i += kNormThreads) cs[i] = turn_cos_sin(a.turn, b, tok - b * a.S, i);
}

template <int DT>
__global__ void __launch_bounds__(kNormThreads) rope_norm_fwd_general_kernel(NormArgs a)
{
    __shared__ float2 cs[ROPE_D_LIMIT / 2];
    __shared__ float rows[kNormWaves][ROPE_D_LIMIT];
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float* z = rows[wave];
    for (uint32_t tok = blockIdx.x; tok < a.tokens; tok += gridDim.x) {
        if (a.rotate) norm_turns(a, tok, cs);      // (the rows of the token before are done)
        const uint32_t b = fast_div(tok, a.s_div), s = tok - b * a.S;
        for (int kind = 0; kind < 2; ++kind) {
            const Rows& x = a.x[kind];
            const Rows& y = a.y[kind];
            for (uint32_t n0 = 0; n0 < a.N[kind]; n0 += kNormWaves) {
                const uint32_t n = n0 + wave;
                const bool live = n < a.N[kind];
                float ss = 0.0f;
                if (live)
                    for (uint32_t j = lane; j < a.D; j += 64) {
                        const float v = Store<DT>::load1(x.data, b * x.sb + s * x.ss + n * x.sn + j);
                        z[j] = v;
                        ss = __builtin_fmaf(v, v, ss);
                    }
                const float r = rsqrtf(__builtin_fmaf(lanes_sum(ss, 64), a.inv_d, a.eps));
                __syncthreads();
                if (live)
                    for (uint32_t j = lane; j < a.D; j += 64) {
                        float v = z[j] * r * norm_weight(a, kind, j);
                        if (a.rotate && j >= a.turn.start && j < a.turn.start + a.turn.L) {
                            bool first;
                            const uint32_t i = turn_pair(a.turn, j - a.turn.start, &first);
                            const uint32_t p = first ? j + a.turn.half : j - a.turn.half;
                            v = rotate_own_unfused(v, z[p] * r * norm_weight(a, kind, p), cs[i].x, cs[i].y, first);
                        }
                        Store<DT>::store1(y.data, b * y.sb + s * y.ss + n * y.sn + j, v);
                    }
                __syncthreads();
            }
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(kNormThreads) rope_norm_bwd_general_kernel(NormArgs a)
{
    __shared__ float2 cs[ROPE_D_LIMIT / 2];
    __shared__ float rows[kNormWaves][ROPE_D_LIMIT];
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float* z = rows[wave];
    for (int kind = 0; kind < 2; ++kind) {
        const Rows& x = a.x[kind];
        const Rows& y = a.y[kind];
        const Rows& dy = a.dy[kind];
        float dw[kNormLanes] = {};
        for (uint32_t tok = blockIdx.x; tok < a.tokens; tok += gridDim.x) {
            if (a.N[kind] == 0) break;
            if (a.rotate) norm_turns(a, tok, cs);
            const uint32_t b = fast_div(tok, a.s_div), s = tok - b * a.S;
            for (uint32_t n0 = 0; n0 < a.N[kind]; n0 += kNormWaves) {
                const uint32_t n = n0 + wave;
                const bool live = n < a.N[kind];
                if (live)
                    for (uint32_t j = lane; j < a.D; j += 64)
                        z[j] = Store<DT>::load1(dy.data, b * dy.sb + s * dy.ss + n * dy.sn + j);
                __syncthreads();
                float v[kNormLanes], g[kNormLanes], ss = 0.0f, dot = 0.0f;
#pragma unroll
                for (int k = 0; k < kNormLanes; ++k) {
                    const uint32_t j = k * 64 + lane;
                    v[k] = g[k] = 0.0f;
                    if (!live || j >= a.D) continue;
                    v[k] = Store<DT>::load1(x.data, b * x.sb + s * x.ss + n * x.sn + j);
                    g[k] = z[j];
                    if (a.rotate && j >= a.turn.start && j < a.turn.start + a.turn.L) {
                        bool first;
                        const uint32_t i = turn_pair(a.turn, j - a.turn.start, &first);
                        g[k] = rotate_own_unfused(g[k], z[first ? j + a.turn.half : j - a.turn.half], cs[i].x, cs[i].y, !first);
                    }
                    ss = __builtin_fmaf(v[k], v[k], ss);
                    dot = __builtin_fmaf(g[k] * norm_weight(a, kind, j), v[k], dot);
                }
                const float r = rsqrtf(__builtin_fmaf(lanes_sum(ss, 64), a.inv_d, a.eps));
                const float m = lanes_sum(dot, 64) * r * a.inv_d;
#pragma unroll
                for (int k = 0; k < kNormLanes; ++k) {
                    const uint32_t j = k * 64 + lane;
                    if (!live || j >= a.D) continue;
                    const float nj = v[k] * r;
                    dw[k] = __builtin_fmaf(g[k], nj, dw[k]);
                    Store<DT>::store1(y.data, b * y.sb + s * y.ss + n * y.sn + j,
                                      r * (g[k] * norm_weight(a, kind, j) - nj * m));
                }
                __syncthreads();
            }
        }
        if (a.part == nullptr) continue;
#pragma unroll
        for (int k = 0; k < kNormLanes; ++k)
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

// The weights' gradients: the blocks' sums added in a fixed order, rounded
// once. A block takes 16 lanes of one weight, 64 strands of partial sums.
struct NormWeightArgs {
    const float* part;
    void* dw[2];
    uint32_t blocks, D;
    int32_t wdt;
};

constexpr int kStrands = 64;

__global__ void __launch_bounds__(1024) rope_norm_weight_grad_kernel(NormWeightArgs a)
{
    __shared__ float sums[kStrands][16];
    const uint32_t strand = threadIdx.x >> 4, l = threadIdx.x & 15, j = blockIdx.x * 16 + l;
    const int kind = blockIdx.y;
    if (a.dw[kind] == nullptr) return;
    float sum = 0.0f;
    if (j < a.D)
        for (uint32_t b = strand; b < a.blocks; b += kStrands) sum += a.part[((uint64_t)b * 2 + kind) * a.D + j];
    sums[strand][l] = sum;
    __syncthreads();
    if (strand != 0 || j >= a.D) return;
    for (int k = 1; k < kStrands; ++k) sum += sums[k][l];
    switch (a.wdt) {
    case ROPE_DTYPE_F32: Store<ROPE_DTYPE_F32>::store1(a.dw[kind], j, sum); break;
    case ROPE_DTYPE_F16: Store<ROPE_DTYPE_F16>::store1(a.dw[kind], j, sum); break;
    default: Store<ROPE_DTYPE_BF16>::store1(a.dw[kind], j, sum); break;
    }
}

}  // namespace
}  // namespace rope
