// The norms of Q's and K's heads with the rotation in the same pass.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <string>

#include "rope_norm_kernels.hpp"
#include "rope_norm_plan.hpp"
#include "rope_rows_host.hpp"

namespace rope {
namespace {

// Blocks of the general forward: what the card holds at a time.
constexpr uint32_t kNormFwdBlocks = 2048;

NormArgs norm_args(const NormPlan& p)
{
    NormArgs a{};
    for (int i = 0; i < 2; ++i) {
        a.x[i] = rows_of(p.x[i]);
        a.y[i] = rows_of(p.y[i]);
        a.dy[i] = rows_of(p.dy[i]);
        a.w[i] = p.w[i];
        a.N[i] = (uint32_t)p.x[i].N;
    }
    a.D = (uint32_t)p.rope.D;
    a.tokens = (uint32_t)(p.B * p.S);
    a.S = (uint32_t)p.S;
    a.wdt = p.wdtype;
    a.eps = p.eps;
    a.inv_d = 1.0f / (float)a.D;
    a.rotate = p.rotate ? 1 : 0;
    a.part = p.part;
    a.turn = turn_of(p.rope);
    if (!p.rotate) a.turn.L = a.turn.pairs = 0;
    a.s_div = make_fastdiv(a.S);
    return a;
}

template <template <int> class K>
const void* by_type(int dtype)
{
    switch (dtype) {
    case ROPE_DTYPE_F32: return K<ROPE_DTYPE_F32>::ptr();
    case ROPE_DTYPE_F16: return K<ROPE_DTYPE_F16>::ptr();
    default: return K<ROPE_DTYPE_BF16>::ptr();
    }
}

template <int NL>
struct General {
    template <int DT>
    struct Fwd {
        static const void* ptr() { return reinterpret_cast<const void*>(&rope_norm_fwd_general_kernel<DT, NL>); }
    };
    template <int DT>
    struct Bwd {
        static const void* ptr() { return reinterpret_cast<const void*>(&rope_norm_bwd_general_kernel<DT, NL>); }
    };
};
template <int NL>
const void* general_kernel(int dtype, bool backward)
{
    return backward ? by_type<General<NL>::template Bwd>(dtype) : by_type<General<NL>::template Fwd>(dtype);
}
const void* norm_general(const NormPlan& p, bool backward)
{
    return p.rope.D <= kNormFewLanes * 64 ? general_kernel<kNormFewLanes>(p.rope.dtype, backward)
                                          : general_kernel<kNormLanes>(p.rope.dtype, backward);
}
template <int C, int PAR>
struct Vec {
    template <int DT>
    struct Fwd {
        static const void* ptr() { return reinterpret_cast<const void*>(&rope_norm_fwd_kernel<DT, C, PAR>); }
    };
    template <int DT>
    struct Bwd {
        static const void* ptr() { return reinterpret_cast<const void*>(&rope_norm_bwd_kernel<DT, C, PAR>); }
    };
};

template <int C, int PAR>
const void* vec_kernel(int dtype, bool backward)
{
    return backward ? by_type<Vec<C, PAR>::template Bwd>(dtype) : by_type<Vec<C, PAR>::template Fwd>(dtype);
}

// The vector kernel of a call, its arguments and LDS; NULL if rows or the slice
// are not in whole chunks.
const void* norm_vec(const NormPlan& p, bool backward, NormVecArgs* a, size_t* lds)
{
    const int es = p.rope.esize;
    for (int i = 0; i < 2; ++i)
        if ((p.w[i] != nullptr && !aligned16(p.w[i])) || !rows_in_chunks(p.x[i], es) || !rows_in_chunks(p.y[i], es) ||
            (backward && !rows_in_chunks(p.dy[i], es)))
            return nullptr;
    if (p.rotate && !turn_in_chunks(p.rope)) return nullptr;
    // Threads per row and chunks per thread: the fewest idle lanes; among those
    // two chunks where that leaves a row 8 threads (128 bytes of 16-bit lanes a
    // load) and forward. (2 x 8191 tokens of 36 heads of 128 lanes, forward: 58
    // us, by one chunk 72; 4 x 4096 of 40 heads, forward and backward: 191, by
    // two chunks both ways 209, by one 196.)
    const uint32_t chunks = a->D / 8;
    uint32_t best = ~0u;
    int C = 1;
    for (uint32_t c = 1; c <= 2; ++c) {
        const uint32_t T = 1u << log2_of((chunks + c - 1) / c);
        if (T > 64) continue;
        const uint32_t cost = 2 * T * c + (T < 8 ? 1 : 0);
        if (cost < best || (cost == best && T >= 8 && !backward)) {
            best = cost;
            a->T = T;
            C = (int)c;
        }
    }
    a->rows_per_block = kNormThreads / a->T;
    const bool own = C == 2 && p.rope.start == 0 && p.rope.half == 8 * (int64_t)a->T && p.rope.L == 2 * p.rope.half;
    // Tokens of a block: as many as leave 1024 blocks (cos and sin then keep
    // more of its threads busy, and K's rows fill it), up to 8. (2 x 8191 tokens:
    // 58 us, by single tokens 103; 32 tokens: 5.3, by eights 10.6.) Fewer tokens
    // than that: a token's heads to as many blocks as its rows fill. (4 tokens of
    // 128 + 16 heads: 5.2 us, a block a token 6.9.)
    uint32_t per = 1;
    while (per < 8 && a->tokens / (2 * per) >= 1024) per *= 2;
    a->tokens_per_block = per;
    a->groups = (a->tokens + per - 1) / per;
    const uint32_t most = std::max(a->N[0], a->N[1]);
    a->splits = backward || per > 1 || a->tokens >= 1024 ? 1 : std::max<uint32_t>(1, (most + a->rows_per_block - 1) / a->rows_per_block);
    a->lds_floats = per * a->turn.pairs;
    *lds = std::max<size_t>(2 * (size_t)a->lds_floats, backward ? (size_t)kNormWaves * a->T * 8 : 0) * sizeof(float);
    a->t_div = make_fastdiv(a->T);
    for (int i = 0; i < 2; ++i) a->n_div[i] = make_fastdiv(std::max<uint32_t>(1, a->N[i]));
    a->pairs_div = make_fastdiv(std::max<uint32_t>(1, a->turn.pairs));
    a->splits_div = make_fastdiv(a->splits);
    // (rows of a block's tokens fit 31 bits, as all rows do)
    if ((uint64_t)a->groups * a->splits > kMaxGridItems / kNormThreads) return nullptr;
    const int par = a->turn.L == 0 || a->turn.half == 1 ? kParNear : own ? kParOwn : kParLoad;
    if (C == 1) return par == kParNear ? vec_kernel<1, kParNear>(p.rope.dtype, backward) : vec_kernel<1, kParLoad>(p.rope.dtype, backward);
    return par == kParNear  ? vec_kernel<2, kParNear>(p.rope.dtype, backward)
           : par == kParOwn ? vec_kernel<2, kParOwn>(p.rope.dtype, backward)
                            : vec_kernel<2, kParLoad>(p.rope.dtype, backward);
}

hipError_t launch_fwd(const NormPlan& p, hipStream_t s)
{
    NormVecArgs a{};
    static_cast<NormArgs&>(a) = norm_args(p);
    size_t lds = 0;
    if (const void* fn = norm_vec(p, false, &a, &lds)) {
        void* args[] = {&a};
        return hipLaunchKernel(fn, dim3(a.groups * a.splits), dim3(kNormThreads), args, lds, s);
    }
    NormArgs g = a;
    void* args[] = {&g};
    const uint32_t blocks = std::min<uint32_t>(g.tokens, kNormFwdBlocks);
    return hipLaunchKernel(norm_general(p, false), dim3(blocks), dim3(kNormThreads), args, 0, s);
}

hipError_t launch_bwd(const NormPlan& p, hipStream_t s)
{
    uint32_t blocks = 0;
    if (!p.noop) {
        NormVecArgs a{};
        static_cast<NormArgs&>(a) = norm_args(p);
        size_t lds = 0;
        const void* fn = norm_vec(p, true, &a, &lds);
        NormArgs g = a;
        void* args[] = {fn != nullptr ? (void*)&a : (void*)&g};
        blocks = (uint32_t)std::min<uint64_t>(fn != nullptr ? a.groups : a.tokens, kNormBwdBlocks);
        hipError_t err = hipLaunchKernel(fn != nullptr ? fn : norm_general(p, true), dim3(blocks), dim3(kNormThreads),
                                         args, fn != nullptr ? lds : 0, s);
        if (err != hipSuccess) return err;
    }
    if (p.dw[0] == nullptr && p.dw[1] == nullptr) return hipSuccess;
    NormWeightArgs w{p.part, {p.dw[0], p.dw[1]}, blocks, (uint32_t)p.rope.D, p.wdtype};
    void* args[] = {&w};
    return hipLaunchKernel(reinterpret_cast<const void*>(&rope_norm_weight_grad_kernel), dim3((w.D + 3) / 4, 2), dim3(kStrands),
                           args, 0, s);
}

}  // namespace
}  // namespace rope

extern "C" {

int64_t rope_qk_norm_workspace(int64_t D) { return rope::norm_workspace_bytes(D); }

rope_status_t rope_qk_norm_fwd(
    int64_t B, int64_t S, rope_dtype_t dtype, const rope_rows_t* q_out, const rope_rows_t* k_out, const rope_rows_t* q,
    const rope_rows_t* k, const void* q_weight, const void* k_weight, rope_dtype_t weight_dtype, double eps,
    const int64_t* positions, const int64_t positions_shape[3], const int64_t positions_strides[3],
    const double* inv_freq, const int32_t* pair_axes, rope_dtype_t table_dtype, int64_t mode,
    const int64_t partial_slice[2], void* stream)
{
    rope::NormPlan p;
    std::string why;
    const rope::Positions in{positions, positions_shape, positions_strides, inv_freq, true, pair_axes, true};
    rope::NormIn qi, ki;
    qi.y = q_out;
    qi.x = q;
    qi.w = q_weight;
    ki.y = k_out;
    ki.x = k;
    ki.w = k_weight;
    rope_status_t st = rope::make_norm_plan(B, S, dtype, qi, ki, false, weight_dtype, eps, in, table_dtype, mode,
                                            partial_slice, nullptr, 0, &p, &why);
    if (st != ROPE_OK) return rope::set_error(st, why);
    if (p.noop) return ROPE_OK;
    return rope::launched(rope::launch_fwd(p, static_cast<hipStream_t>(stream)));
}

rope_status_t rope_qk_norm_bwd(
    int64_t B, int64_t S, rope_dtype_t dtype, const rope_rows_t* dq, const rope_rows_t* dk, void* dq_weight,
    void* dk_weight, const rope_rows_t* q_grad, const rope_rows_t* k_grad, const rope_rows_t* q, const rope_rows_t* k,
    const void* q_weight, const void* k_weight, rope_dtype_t weight_dtype, double eps, const int64_t* positions,
    const int64_t positions_shape[3], const int64_t positions_strides[3], const double* inv_freq,
    const int32_t* pair_axes, rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2], void* workspace,
    int64_t workspace_bytes, void* stream)
{
    rope::NormPlan p;
    std::string why;
    const rope::Positions in{positions, positions_shape, positions_strides, inv_freq, true, pair_axes, true};
    const rope::NormIn qi{dq, q, q_grad, q_weight, dq_weight}, ki{dk, k, k_grad, k_weight, dk_weight};
    rope_status_t st = rope::make_norm_plan(B, S, dtype, qi, ki, true, weight_dtype, eps, in, table_dtype, mode,
                                            partial_slice, workspace, workspace_bytes, &p, &why);
    if (st != ROPE_OK) return rope::set_error(st, why);
    return rope::launched(rope::launch_bwd(p, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
