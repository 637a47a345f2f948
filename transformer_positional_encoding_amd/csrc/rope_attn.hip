// Attention of new tokens over a paged cache held in 4 bits.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <string>

#include "rope_attn_kernels.hpp"
#include "rope_attn_plan.hpp"
#include "rope_rows_host.hpp"

namespace rope {
namespace {

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
struct General {
    static const void* ptr() { return reinterpret_cast<const void*>(&rope_attn_general_kernel<DT>); }
};
template <int DT>
struct Join {
    static const void* ptr() { return reinterpret_cast<const void*>(&rope_attn_join_kernel<DT>); }
};

AttnArgs attn_args(const AttnPlan& p)
{
    AttnArgs a{};
    a.q = rows_of(p.q);
    a.out = rows_of(p.out);
    a.kc = cache_of(p.kc);
    a.vc = cache_of(p.vc);
    a.D = (uint32_t)p.q.D;
    a.Dv = (uint32_t)p.out.D;
    a.S = (uint32_t)p.S;
    a.Hq = (uint32_t)p.q.N;
    a.heads = (uint32_t)p.heads;
    a.rep = (uint32_t)p.rep;
    a.rows = (uint32_t)(p.S * p.rep);
    a.splits = (uint32_t)p.splits;
    a.table = p.table;
    a.table_stride = p.table_stride;
    a.lengths = p.lengths;
    a.counts = p.counts;
    a.pages = p.pages;
    a.most = (int32_t)p.most;
    // (no token number reaches 2^31 - 1, so a page of as many or more holds all)
    a.page_div = make_fastdiv((uint32_t)std::min<int64_t>(p.page_size, INT32_MAX));
    a.scale2 = (float)(p.scale * 1.4426950408889634);
    a.causal = p.causal ? 1 : 0;
    a.part = p.part;
    a.part_rows = (uint64_t)p.B * (uint64_t)p.S * (uint64_t)p.q.N;
    a.rep_div = make_fastdiv(a.rep);
    a.heads_div = make_fastdiv(a.heads);
    a.splits_div = make_fastdiv(a.splits);
    return a;
}

rope_status_t launch_attn(const AttnPlan& p, hipStream_t s)
{
    AttnArgs a = attn_args(p);
    void* args[] = {&a};
    a.tiles = (a.rows + kAttnGenRows - 1) / kAttnGenRows;
    a.tiles_div = make_fastdiv(a.tiles);
    const uint64_t blocks = (uint64_t)p.B * a.heads * a.tiles * a.splits;
    if (blocks >= (1ull << 31) || blocks > kMaxGridItems / kAttnGenThreads)
        return set_error(ROPE_ERR_UNSUPPORTED, "a grid too large for one launch");
    hipError_t err = hipLaunchKernel(by_type<General>(p.rope.dtype), dim3((uint32_t)blocks), dim3(kAttnGenThreads), args, 0, s);
    if (err != hipSuccess || a.splits == 1) return launched(err);
    return launched(hipLaunchKernel(by_type<Join>(p.rope.dtype), dim3((uint32_t)((a.part_rows + 3) / 4)), dim3(256), args, 0, s));
}

}  // namespace
}  // namespace rope

extern "C" {

int64_t rope_cache_attention_workspace(int64_t B, int64_t S, int64_t q_heads, int64_t heads, int64_t Dv)
{
    return rope::attn_workspace_bytes(B, S, q_heads, heads, Dv);
}

rope_status_t rope_cache_attention(
    int64_t B, int64_t S, rope_dtype_t dtype, const rope_rows_t* out, const rope_rows_t* q, const rope_cache_t* k_cache,
    const rope_cache_t* v_cache, const int32_t* block_table, int64_t table_pages, int64_t table_stride,
    const int32_t* lengths, const int32_t* counts, double scale, int32_t causal, void* workspace,
    int64_t workspace_bytes, void* stream)
{
    rope::AttnPlan p;
    std::string why;
    rope_status_t st = rope::make_attn_plan(B, S, dtype, out, q, k_cache, v_cache, block_table, table_pages, table_stride,
                                            lengths, counts, scale, causal != 0, workspace, workspace_bytes, &p, &why);
    if (st != ROPE_OK) return rope::set_error(st, why);
    if (p.noop) return ROPE_OK;
    return rope::launch_attn(p, static_cast<hipStream_t>(stream));
}

}  // extern "C"
