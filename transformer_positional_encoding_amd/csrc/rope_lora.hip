// rope_proj_lora_fwd: a head projection shared by many requests, each token
// with its own low-rank adapter, and a rotary epilogue.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <string>

#include "rope_host.hpp"
#include "rope_lora_kernels.hpp"
#include "rope_plan.hpp"

namespace rope {
namespace {

constexpr uint64_t kMaxGridItems = 0xFFFFFFFFull;   // work-items of a launch

struct LoraLaunch {
    ProjPlan q;
    LoraProjArgs g{};
    int tdt = ROPE_DTYPE_BF16;
    int heads = 0;
};

rope_status_t prepare_lora(void* y, rope_dtype_t y_dtype, const void* x, const void* w, rope_dtype_t dtype,
                           const int64_t y_shape[4], int64_t K, const rope_lora_t* lora,
                           const void* r1, const int64_t r1_shape[4], const int64_t r1_strides[4],
                           const void* r2, const int64_t r2_shape[4], const int64_t r2_strides[4],
                           rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2], void* workspace,
                           int64_t workspace_bytes, LoraLaunch* P, std::string* why)
{
    const LoraCheck c{lora, workspace, workspace_bytes};
    rope_status_t st = make_proj_plan(y, y_dtype, x, w, dtype, y_shape, K, r1, r1_shape, r1_strides, r2, r2_shape,
                                      r2_strides, table_dtype, mode, partial_slice, &P->q, why, &c);
    if (st != ROPE_OK || P->q.noop) return st;
    const Plan& p = P->q.rope;
    ProjArgs& a = P->g.p;
    a.x = static_cast<const uint16_t*>(P->q.x);
    a.w = static_cast<const uint16_t*>(P->q.w);
    a.y = P->q.y;
    a.ydt = P->q.out_dtype;
    a.r1 = p.r1;
    a.r2 = p.r2;
    a.t1b = p.t1[0]; a.t1s = p.t1[1]; a.t1n = p.t1[2];
    a.t2b = p.t2[0]; a.t2s = p.t2[1]; a.t2n = p.t2[2];
    a.M = (int32_t)(p.B * p.S);
    a.N = (int32_t)(p.N * p.D);
    a.K = (int32_t)P->q.K;
    a.S = (int32_t)p.S;
    a.Dh = (int32_t)p.D;
    a.start = (int32_t)p.start;
    a.L = (int32_t)p.L;
    a.half = p.L > 0 ? (int32_t)p.half : 1;
    a.s_div = make_fastdiv((uint32_t)p.S);
    a.dh_div = make_fastdiv((uint32_t)p.D);
    P->tdt = p.L > 0 ? p.tdtype : (int)ROPE_DTYPE_BF16;
    P->heads = (int)p.N;
    LoraArgs& l = P->g.l;
    if (lora->count > 0 && lora->rank > 0) {
        l.a = static_cast<const uint16_t*>(lora->a);
        l.b = static_cast<const uint16_t*>(lora->b);
        l.ids = lora->adapters;
        l.scales = lora->scales;
        l.h = static_cast<float*>(workspace);
        l.count = (int32_t)lora->count;
        l.R = (int32_t)lora->rank;
    }
    return ROPE_OK;
}

template <int DT>
hipError_t launch_lora(const LoraLaunch& P, hipStream_t s)
{
    const ProjArgs& a = P.g.p;
    const LoraArgs& l = P.g.l;
    if (l.count > 0) {
        const uint32_t gy = (uint32_t)(l.R + kShrinkWaves - 1) / kShrinkWaves;
        const uint32_t gx = (uint32_t)std::min<uint64_t>((uint64_t)a.M, kMaxGridItems / (64 * kShrinkWaves) / gy);
        hipLaunchKernelGGL((rope_lora_shrink_kernel<DT>), dim3(gx, gy), dim3(64 * kShrinkWaves), 0, s, l, a.x, a.M, a.K);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    const uint64_t tiles = (uint64_t)((a.M + kHeadTokens - 1) / kHeadTokens) * (uint64_t)P.heads;
    hipLaunchKernelGGL((rope_lora_head_kernel<DT>), dim3((uint32_t)std::min<uint64_t>(tiles, kMaxGridItems / 256)),
                       dim3(256), 0, s, P.g, P.tdt, P.heads);
    return hipGetLastError();
}

}  // namespace
}  // namespace rope

extern "C" {

rope_status_t rope_proj_lora_fwd(
    void* y, rope_dtype_t y_dtype, const void* x, const void* w, rope_dtype_t dtype,
    const int64_t y_shape[4], int64_t K, const rope_lora_t* lora,
    const void* r1, const int64_t r1_shape[4], const int64_t r1_strides[4],
    const void* r2, const int64_t r2_shape[4], const int64_t r2_strides[4],
    rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* workspace, int64_t workspace_bytes, void* stream)
{
    rope::LoraLaunch P;
    std::string why;
    rope_status_t st = rope::prepare_lora(y, y_dtype, x, w, dtype, y_shape, K, lora, r1, r1_shape, r1_strides, r2,
                                          r2_shape, r2_strides, table_dtype, mode, partial_slice, workspace,
                                          workspace_bytes, &P, &why);
    if (st != ROPE_OK) return rope::set_error(st, why);
    if (P.q.noop) return ROPE_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t err = P.q.in_dtype == ROPE_DTYPE_BF16 ? rope::launch_lora<ROPE_DTYPE_BF16>(P, s)
                                                           : rope::launch_lora<ROPE_DTYPE_F16>(P, s);
    if (err != hipSuccess)
        return rope::set_error(ROPE_ERR_RUNTIME, std::string("kernel launch: ") + hipGetErrorString(err));
    return ROPE_OK;
}

int64_t rope_proj_lora_workspace(const int64_t y_shape[4], int64_t K, int64_t rank)
{
    if (y_shape == nullptr || K <= 0 || rank <= 0 || rank > ROPE_LORA_RANK_MAX || y_shape[0] <= 0 || y_shape[1] <= 0)
        return 0;
    int64_t M;
    if (__builtin_mul_overflow(y_shape[0], y_shape[1], &M)) return 0;
    const int64_t n = rope::lora_workspace_bytes(M, rank);
    return n < 0 ? 0 : n;
}

}  // extern "C"
