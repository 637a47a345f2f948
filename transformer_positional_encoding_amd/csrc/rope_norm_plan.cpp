// Argument checking of the norms of Q's and K's heads (see rope_norm_plan.hpp).
#include "rope_norm_plan.hpp"

#include <cmath>

namespace rope {

int64_t norm_workspace_bytes(int64_t D) { return D <= 0 || D > ROPE_D_LIMIT ? 0 : kNormBwdBlocks * 2 * D * 4; }

rope_status_t make_norm_plan(int64_t B, int64_t S, rope_dtype_t dtype, const NormIn& q, const NormIn& k, bool backward,
                             rope_dtype_t weight_dtype, double eps, const Positions& in, rope_dtype_t table_dtype,
                             int64_t mode, const int64_t partial_slice[2], void* workspace, int64_t workspace_bytes,
                             NormPlan* plan, std::string* why)
{
    NormPlan p;
    const char* const out_name[2] = {backward ? "dq" : "q_out", backward ? "dk" : "k_out"};
    const char* const in_name[2] = {"q", "k"};
    const char* const grad_name[2] = {"q_grad", "k_grad"};
    const NormIn* const side[2] = {&q, &k};
    if (q.x == nullptr || q.y == nullptr || (backward && q.dy == nullptr))
        return fail(ROPE_ERR_NULLPTR, why, std::string("q, ") + out_name[0] + (backward ? " or q_grad" : "") + " is NULL");
    if ((k.x == nullptr) != (k.y == nullptr) || (backward && (k.x == nullptr) != (k.dy == nullptr)))
        return fail(ROPE_ERR_NULLPTR, why, "k and what goes with it must all be given or all be NULL");
    rope_status_t st = make_plan_scalars(B, S, q.x->N, q.x->D, dtype, table_dtype, mode, partial_slice, &p.rope, why);
    if (st != ROPE_OK) return st;
    const int es = p.rope.esize;
    const int64_t D = q.x->D;
    if (weight_dtype < ROPE_DTYPE_F32 || weight_dtype > ROPE_DTYPE_BF16)
        return fail(ROPE_ERR_INVALID, why, "unknown weight_dtype");
    if (!(eps >= 0) || !std::isfinite(eps)) return fail(ROPE_ERR_INVALID, why, "eps must be finite and not negative");
    p.B = B;
    p.S = S;
    p.wdtype = (int)weight_dtype;
    p.eps = (float)eps;
    int64_t tokens, rows = 0;
    if (__builtin_mul_overflow(B, S, &tokens)) return fail(ROPE_ERR_INVALID, why, "more rows than 64-bit offsets can address");
    for (int i = 0; i < 2; ++i) {
        const NormIn& s = *side[i];
        if (s.x == nullptr) continue;
        if (s.x->N < 0) return fail(ROPE_ERR_INVALID, why, std::string(in_name[i]) + ": negative dimension");
        if (s.x->D != D) return fail(ROPE_ERR_INVALID, why, "k: its lanes must be q's");
        const rope_rows_t* others[2] = {s.y, backward ? s.dy : nullptr};
        const char* names[2] = {out_name[i], grad_name[i]};
        for (int j = 0; j < 2; ++j)
            if (others[j] != nullptr && (others[j]->N != s.x->N || others[j]->D != D))
                return fail(ROPE_ERR_INVALID, why, std::string(names[j]) + ": its heads and lanes must be " + in_name[i] + "'s");
        if ((st = check_rows(in_name[i], *s.x, B, S, es, false, &p.x[i], why)) != ROPE_OK) return st;
        if ((st = check_rows(out_name[i], *s.y, B, S, es, true, &p.y[i], why)) != ROPE_OK) return st;
        if (backward && (st = check_rows(grad_name[i], *s.dy, B, S, es, false, &p.dy[i], why)) != ROPE_OK) return st;
        int64_t n;
        if (__builtin_mul_overflow(tokens, s.x->N, &n) || __builtin_add_overflow(rows, n, &rows))
            return fail(ROPE_ERR_INVALID, why, "more rows than 64-bit offsets can address");
        if (s.dw != nullptr && s.w == nullptr)
            return fail(ROPE_ERR_INVALID, why, "a weight that is not there has no gradient");
        p.w[i] = s.w;
        p.dw[i] = s.dw;
        const uintptr_t ws = (uintptr_t)element_size((int)weight_dtype);
        if (reinterpret_cast<uintptr_t>(s.w) % ws != 0 || reinterpret_cast<uintptr_t>(s.dw) % ws != 0)
            return fail(ROPE_ERR_INVALID, why, "weights and their gradients must be aligned to their elements");
    }
    if (rows >= (1ll << 31)) return fail(ROPE_ERR_UNSUPPORTED, why, "2^31 rows of q and k or more");
    p.noop = rows == 0 || D == 0;
    if (D == 0) p.dw[0] = p.dw[1] = nullptr;
    if (!p.noop) {
        for (int i = 0; i < 2; ++i) {
            if (p.x[i].N == 0) continue;
            if ((st = check_data(in_name[i], p.x[i], es, why)) != ROPE_OK) return st;
            if ((st = check_data(out_name[i], p.y[i], es, why)) != ROPE_OK) return st;
            if (backward && (st = check_data(grad_name[i], p.dy[i], es, why)) != ROPE_OK) return st;
        }
        if (p.dw[0] != nullptr || p.dw[1] != nullptr) {
            if (workspace == nullptr) return fail(ROPE_ERR_NULLPTR, why, "workspace is NULL");
            if (reinterpret_cast<uintptr_t>(workspace) % 16 != 0)
                return fail(ROPE_ERR_INVALID, why, "workspace must be 16-byte aligned");
            if (workspace_bytes < norm_workspace_bytes(D)) return fail(ROPE_ERR_INVALID, why, "workspace too small");
            p.part = static_cast<float*>(workspace);
        }
        p.rotate = in.data != nullptr && p.rope.L > 0;
        if (p.rotate && (st = check_positions(B, S, p.rope.L, in, &p.rope, why)) != ROPE_OK) return st;
    }
    *plan = p;
    return ROPE_OK;
}

}  // namespace rope
