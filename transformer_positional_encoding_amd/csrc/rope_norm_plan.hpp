// Host-side checks of the norms of Q's and K's heads (rope_qk_norm_fwd,
// rope_qk_norm_bwd). Pure C++ (no HIP), so they run without a GPU.
#pragma once

#include "rope_cache_plan.hpp"

namespace rope {

// What a call is given of Q or K. Backward: dy the incoming gradient, y the
// rows that take x's gradient, dw what takes the weight's.
struct NormIn {
    const rope_rows_t* y = nullptr;
    const rope_rows_t* x = nullptr;
    const rope_rows_t* dy = nullptr;
    const void* w = nullptr;
    void* dw = nullptr;
};

struct NormPlan {
    Plan rope;                  // the slice, mode and positions; D
    int64_t B = 0, S = 0;
    RowsPlan x[2], y[2], dy[2];   // of Q and of K; N 0: none
    const void* w[2] = {nullptr, nullptr};
    void* dw[2] = {nullptr, nullptr};
    int wdtype = 0;
    float eps = 0;
    bool rotate = false;
    bool noop = false;          // no rows (backward: the weights' gradients are 0)
    float* part = nullptr;      // backward: the weights' partial sums
};

// Blocks of the backward pass: each leaves a sum of D floats for each of the
// two weights.
constexpr int64_t kNormBwdBlocks = 1024;

// Bytes of workspace of a backward call.
int64_t norm_workspace_bytes(int64_t D);

rope_status_t make_norm_plan(int64_t B, int64_t S, rope_dtype_t dtype, const NormIn& q, const NormIn& k, bool backward,
                             rope_dtype_t weight_dtype, double eps, const Positions& in, rope_dtype_t table_dtype,
                             int64_t mode, const int64_t partial_slice[2], void* workspace, int64_t workspace_bytes,
                             NormPlan* plan, std::string* why);

}  // namespace rope
