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

template <int DT>
struct FwdGeneral {
    static const void* ptr() { return reinterpret_cast<const void*>(&rope_norm_fwd_general_kernel<DT>); }
};
template <int DT>
struct BwdGeneral {
    static const void* ptr() { return reinterpret_cast<const void*>(&rope_norm_bwd_general_kernel<DT>); }
};

hipError_t launch_fwd(const NormPlan& p, hipStream_t s)
{
    NormArgs a = norm_args(p);
    void* args[] = {&a};
    const uint32_t blocks = (uint32_t)std::min<uint64_t>(a.tokens, kMaxGridItems / kNormThreads);
    return hipLaunchKernel(by_type<FwdGeneral>(p.rope.dtype), dim3(blocks), dim3(kNormThreads), args, 0, s);
}

hipError_t launch_bwd(const NormPlan& p, hipStream_t s)
{
    uint32_t blocks = 0;
    if (!p.noop) {
        NormArgs a = norm_args(p);
        void* args[] = {&a};
        blocks = (uint32_t)std::min<uint64_t>(a.tokens, kNormBwdBlocks);
        hipError_t err = hipLaunchKernel(by_type<BwdGeneral>(p.rope.dtype), dim3(blocks), dim3(kNormThreads), args, 0, s);
        if (err != hipSuccess) return err;
    }
    if (p.dw[0] == nullptr && p.dw[1] == nullptr) return hipSuccess;
    NormWeightArgs w{p.part, {p.dw[0], p.dw[1]}, blocks, (uint32_t)p.rope.D, p.wdtype};
    void* args[] = {&w};
    return hipLaunchKernel(reinterpret_cast<const void*>(&rope_norm_weight_grad_kernel), dim3((w.D + 15) / 16, 2), dim3(1024),
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
