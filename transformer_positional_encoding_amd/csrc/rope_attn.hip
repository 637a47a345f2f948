// Attention of new tokens over a paged cache held in 4 bits.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <string>

#include "rope_attn_host.hpp"
#include "rope_attn_mfma_kernels.hpp"
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
struct JoinFew {
    static const void* ptr() { return reinterpret_cast<const void*>(&rope_attn_join_few_kernel<DT>); }
};
template <int DT>
struct JoinMany {
    static const void* ptr() { return reinterpret_cast<const void*>(&rope_attn_join_many_kernel<DT>); }
};

// Whether waves join a row each, of up to kJoinFewParts parts: not where many
// parts meet few rows. (16 parts of 3200 rows: 72 us a call of 16 sequences,
// with a block a row and 32 lanes 135; 64 of 128, 4 sequences of up to 100000
// tokens: 139 and 115.)
bool join_few(const AttnArgs& a)
{
    return a.parts <= 32 * a.B || (a.parts <= 64 * a.B && (uint64_t)a.B * a.part_rows >= 512);
}

// Whether rows of codes start and step at multiples of `bytes`.
bool codes_aligned(const CachePlan& c, uintptr_t bytes)
{
    return reinterpret_cast<uintptr_t>(c.data) % bytes == 0 && c.st[0] % (int64_t)bytes == 0 &&
           c.st[1] % (int64_t)bytes == 0 && c.st[2] % (int64_t)bytes == 0;
}

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
    a.table = p.table;
    a.table_stride = p.table_stride;
    a.lengths = p.lengths;
    a.counts = p.counts;
    a.pages = p.pages;
    a.page_limit = (uint32_t)std::min<int64_t>(p.pages, INT32_MAX);
    a.most = (int32_t)p.most;
    // (no token number reaches 2^31 - 1, so a page of as many or more holds all)
    a.page_div = make_fastdiv((uint32_t)std::min<int64_t>(p.page_size, INT32_MAX));
    a.scale2 = (float)(p.scale * 1.4426950408889634);
    a.causal = p.causal ? 1 : 0;
    a.part = p.part;
    a.part_rows = (uint32_t)(p.S * p.q.N);
    a.B = (uint32_t)p.B;
    a.parts = (uint32_t)p.parts;
    a.split = a.parts > a.B;
    a.most_parts = join_few(a) ? kJoinFewParts : kAttnMaxParts;
    a.unit = kAttnGenThreads;
    a.words = codes_aligned(p.kc, 4) && p.kc.group % 8 == 0 ? 1 : 0;
    a.rep_div = make_fastdiv(a.rep);
    a.heads_div = make_fastdiv(a.heads);
    return a;
}

// Whether the rows of four heads lie beside each other in 16-byte pieces, and
// those of their scales that are one a row.
bool heads_together(const CachePlan& c, int64_t heads, int64_t D, bool scales)
{
    return heads % 4 == 0 && codes_aligned(c, 16) && c.st[2] == D / 2 &&
           (!scales || (aligned16(c.scales) && c.sc[0] % 4 == 0 && c.sc[1] % 4 == 0 && c.sc[2] == 1));
}

// (Four heads loaded together, and by waves on their own: 64 sequences of up to
// 8192 tokens, 32 heads on 8 of 128 lanes 103 and 118 us; 64 heads on 16 of 64
// 148 and 225; scales of 32 lanes 156 and 235; 16 sequences of 5 new tokens, 40
// heads on 8, scales of 32 72 and 102.)

// How the matrix-core kernels for rows of up to `lanes` lanes see a call's
// scales; -1 if they do not take it.
int scales_of(const AttnPlan& p, int lanes)
{
    const int64_t D = p.q.D, Dv = p.out.D;
    if (p.rope.dtype == ROPE_DTYPE_F32 || D > 256 || Dv > 256 || !rows_in_chunks(p.q, 2) || !rows_in_chunks(p.out, 2) ||
        !codes_aligned(p.kc, 4) || !codes_aligned(p.vc, lanes == 64 ? 2 : 4))
        return -1;
    const bool k_row = p.kc.group == D, v_row = p.vc.group == Dv;
    if ((!k_row && p.kc.group % 16 != 0) || (!v_row && p.vc.group % 16 != 0)) return -1;
    const bool k_halves = !k_row && p.kc.group % 32 != 0, v_halves = !v_row && p.vc.group % 32 != 0;
    if (v_halves) return k_halves ? kAttnHalves : kAttnVHalves;
    if (k_halves) return v_row ? kAttnKHalves : kAttnHalves;
    const bool k_whole = k_row && D == lanes && codes_aligned(p.kc, lanes == 64 ? 8 : 16);
    return !v_row ? kAttnSegments : k_whole ? kAttnRowScales : kAttnKSegments;
}

// The matrix-core kernel of a call.
const void* mfma_kernel(const AttnPlan& p, AttnRowsOf rows, bool few, int lanes, int scales, int64_t heads)
{
    const int64_t D = p.q.D, Dv = p.out.D;
    const bool whole16 = p.page_size % 16 == 0 && p.kc.st[1] < (1 << 26) && p.vc.st[1] < (1 << 26);
    if (few && lanes < 256 && whole16 && D == lanes && Dv == lanes &&
        heads_together(p.kc, heads, D, scales == kAttnRowScales) && heads_together(p.vc, heads, D, scales == kAttnRowScales))
        rows = rows == AttnRowsOf::kOneTile ? AttnRowsOf::kFourHeads : AttnRowsOf::kFourHeadsTwoTiles;
    if (p.rope.dtype == ROPE_DTYPE_BF16)
        return whole16 ? attn_kernel_bf16(lanes, scales, rows) : attn_kernel_bf16_any(lanes, scales, rows);
    return whole16 ? attn_kernel_f16(lanes, scales, rows) : attn_kernel_f16_any(lanes, scales, rows);
}

rope_status_t launch_attn(const AttnPlan& p, hipStream_t s)
{
    AttnVecArgs a{};
    static_cast<AttnArgs&>(a) = attn_args(p);
    const int lanes = std::max(p.q.D, p.out.D) <= 64 ? 64 : std::max(p.q.D, p.out.D) <= 128 ? 128 : 256;
    const int scales = scales_of(p, lanes);
    // Rows of a cached head: up to 16 a tile of them a wave; up to 64 two tiles
    // (24 rows, 8 sequences of up to 8000 tokens, 32 heads on 8: 38 us, one tile
    // 49, shared numbers 71; 64 rows 51, 65 and 66); more share their numbers (96
    // rows 75, two tiles 69; 128 rows 79 and 86, 512 rows 247 and 284). Rows past
    // 128 lanes and scales of 16 leave registers for one tile a wave; the latter
    // share their numbers all the same (3 prompts of 2039 tokens behind up to
    // 4096: 2090 us, 3820 by waves on their own), the former do not.
    const bool halves = scales >= kAttnKHalves;
    const AttnRowsOf rows = lanes < 256 && a.rows > 64              ? AttnRowsOf::kShared
                            : lanes < 256 && a.rows > 16 && !halves ? AttnRowsOf::kTwoTiles
                                                                    : AttnRowsOf::kOneTile;
    const bool mfma = scales >= 0;
    const void* fn = mfma ? mfma_kernel(p, rows, a.rows <= 64, lanes, scales, a.heads) : by_type<General>(p.rope.dtype);
    // Up to 64 rows: a wave a head, as far as heads go by fours, which then read
    // neighbouring bytes; else waves take turns at the tokens. More: a wave its
    // own rows.
    a.head_waves = a.token_waves = a.row_waves = 1;
    if (a.rows > 64) a.row_waves = 4;
    else if (a.heads % 4 == 0) a.head_waves = 4;
    else a.token_waves = a.heads % 2 == 0 ? 2 : 4;
    if (a.token_waves == 2) a.head_waves = 2;
    if (mfma) {
        a.heads_div = make_fastdiv(a.heads / a.head_waves);
        a.unit = 64 * (a.row_waves > 1 ? 1 : a.token_waves);
    }
    a.k_group = a.kc.group;
    a.v_group = a.vc.group;
    a.k_groups = a.D / a.k_group;
    a.v_groups = a.Dv / a.v_group;
    const uint32_t block_rows = !mfma ? kAttnGenRows : (rows == AttnRowsOf::kOneTile || halves ? 16 : 32) * a.row_waves;
    a.tiles = (a.rows + block_rows - 1) / block_rows;
    a.tiles_div = make_fastdiv(a.tiles);
    const uint64_t blocks = (uint64_t)a.parts * a.heads_div.d * a.tiles;
    if (blocks >= (1ull << 31) || blocks > kMaxGridItems / kAttnGenThreads)
        return set_error(ROPE_ERR_UNSUPPORTED, "a grid too large for one launch");
    AttnArgs g = a;
    void* args[] = {mfma ? (void*)&a : (void*)&g};
    hipError_t err = hipLaunchKernel(fn, dim3((uint32_t)blocks), dim3(kAttnGenThreads),
                                     args, 0, s);
    if (err != hipSuccess || !a.split) return launched(err);
    args[0] = &g;
    const uint64_t rows_of_all = (uint64_t)a.B * a.part_rows;
    if (!join_few(a))
        return launched(hipLaunchKernel(by_type<JoinMany>(p.rope.dtype), dim3((uint32_t)rows_of_all, (a.Dv + kJoinLanes - 1) / kJoinLanes),
                                        dim3(kJoinThreads), args, 0, s));
    return launched(hipLaunchKernel(by_type<JoinFew>(p.rope.dtype), dim3((uint32_t)((rows_of_all + kJoinRows - 1) / kJoinRows)),
                                    dim3(kJoinThreads), args, 0, s));
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
