// Argument checking of attention over a paged cache (see rope_attn_plan.hpp).
#include "rope_attn_plan.hpp"

#include <algorithm>
#include <cmath>
#include <limits>

namespace rope {

namespace {

constexpr int64_t kI64Max = std::numeric_limits<int64_t>::max();
// The fewest tokens that are worth a part of their own. (One sequence of 500
// tokens, 4 heads of 64 lanes: 9.1 us by 64, 12.6 by 256; of 4000 10.8 and
// 15.4.)
constexpr int64_t kAttnSplitTokens = 64;

}  // namespace

int64_t attn_parts(int64_t B, int64_t heads, int64_t rows, int64_t tokens)
{
    // up to 64 rows: as many as a wave takes; a block's 128 are worth 8 tiles
    const int64_t tiles = rows <= 16 ? 1 : rows <= 64 ? (rows + 31) / 32 : (rows + 15) / 16;
    const int64_t per_head = heads > kAttnBlocks / tiles ? 0 : kAttnBlocks / (heads * tiles);
    const int64_t parts = std::min(per_head, B * std::min(kAttnMaxParts, tokens / kAttnSplitTokens));
    return B <= kAttnMaxSplit && 4 * parts >= 5 * B ? parts : B;
}

int64_t attn_workspace_bytes(int64_t B, int64_t S, int64_t q_heads, int64_t heads, int64_t Dv)
{
    if (B <= 0 || S <= 0 || q_heads <= 0 || heads <= 0 || q_heads % heads != 0 || Dv <= 0 || Dv > ROPE_D_LIMIT) return 0;
    int64_t rows;
    if (__builtin_mul_overflow(B, S, &rows) || __builtin_mul_overflow(rows, q_heads, &rows) || rows >= (1ll << 31)) return 0;
    const int64_t parts = attn_parts(B, heads, S * (q_heads / heads), kI64Max);
    return parts == B ? 0 : parts * S * q_heads * (Dv + 2) * 4;
}

rope_status_t make_attn_plan(int64_t B, int64_t S, rope_dtype_t dtype, const rope_rows_t* out, const rope_rows_t* q,
                             const rope_cache_t* k_cache, const rope_cache_t* v_cache, const int32_t* block_table,
                             int64_t table_pages, int64_t table_stride, const int32_t* lengths, const int32_t* counts,
                             double scale, bool causal, void* workspace, int64_t workspace_bytes, AttnPlan* plan,
                             std::string* why)
{
    AttnPlan p;
    if (out == nullptr || q == nullptr || k_cache == nullptr || v_cache == nullptr)
        return fail(ROPE_ERR_NULLPTR, why, "out, q, k_cache or v_cache is NULL");
    const int64_t none[2] = {0, 0};
    rope_status_t st = make_plan_scalars(B, S, q->N, q->D, dtype, dtype, ROPE_MODE_ROTATE_HALF, none, &p.rope, why);
    if (st != ROPE_OK) return st;
    const int es = p.rope.esize;
    if ((st = check_cache("k_cache", *k_cache, dtype, false, &p.kc, why)) != ROPE_OK) return st;
    if ((st = check_cache("v_cache", *v_cache, dtype, false, &p.vc, why)) != ROPE_OK) return st;
    if (k_cache->format != ROPE_CACHE_INT4 || v_cache->format != ROPE_CACHE_INT4)
        return fail(ROPE_ERR_UNSUPPORTED, why, "attention reads caches held in 4 bits (ROPE_CACHE_INT4)");
    if (v_cache->pages != k_cache->pages || v_cache->page_size != k_cache->page_size || v_cache->heads != k_cache->heads)
        return fail(ROPE_ERR_INVALID, why, "v_cache: its pages and heads must be k_cache's");
    if (q->D != k_cache->dim) return fail(ROPE_ERR_INVALID, why, "q: its lanes must be k_cache's");
    if (out->D != v_cache->dim || out->N != q->N)
        return fail(ROPE_ERR_INVALID, why, "out: its heads must be q's and its lanes v_cache's");
    if (k_cache->heads < 1 || q->N % k_cache->heads != 0)
        return fail(ROPE_ERR_INVALID, why, "q: its heads must be a multiple of the caches'");
    if (q->D < 2 || out->D < 2) return fail(ROPE_ERR_INVALID, why, "rows without lanes");
    if ((st = check_rows("q", *q, B, S, es, false, &p.q, why)) != ROPE_OK) return st;
    if ((st = check_rows("out", *out, B, S, es, true, &p.out, why)) != ROPE_OK) return st;
    if (table_pages < 0 || table_stride < 0) return fail(ROPE_ERR_INVALID, why, "block_table: negative size or stride");
    const int64_t table_counts[2] = {B, table_pages}, steps[2] = {table_stride, 1};
    const int64_t ext = extent(table_counts, steps, 2, 1);
    if (ext < 0 || ext > kI64Max / 4) return fail(ROPE_ERR_INVALID, why, "block_table: stride overflows 64-bit offsets");
    if (!(scale > 0) || !std::isfinite(scale) || !((float)scale > 0) || !std::isfinite((float)scale))
        return fail(ROPE_ERR_INVALID, why, "scale must be positive and finite");
    p.B = B;
    p.S = S;
    p.heads = k_cache->heads;
    p.rep = q->N / p.heads;
    p.scale = scale;
    p.causal = causal;
    int64_t tokens, rows;
    if (__builtin_mul_overflow(B, S, &tokens) || __builtin_mul_overflow(tokens, q->N, &rows))
        return fail(ROPE_ERR_INVALID, why, "more rows than 64-bit offsets can address");
    if (rows == 0) {
        p.noop = true;
        *plan = p;
        return ROPE_OK;
    }
    if (rows >= (1ll << 31)) return fail(ROPE_ERR_UNSUPPORTED, why, "2^31 rows or more");
    if ((st = check_data("q", p.q, es, why)) != ROPE_OK) return st;
    if ((st = check_data("out", p.out, es, why)) != ROPE_OK) return st;
    if (lengths == nullptr) return fail(ROPE_ERR_NULLPTR, why, "lengths is NULL");
    // a cache without slots, or a table without columns, holds no token: their
    // pointers are not looked at
    if (k_cache->pages > 0 && k_cache->page_size > 0 && table_pages > 0) {
        if ((st = check_pointers("k_cache", p.kc, why)) != ROPE_OK) return st;
        if ((st = check_pointers("v_cache", p.vc, why)) != ROPE_OK) return st;
        if (block_table == nullptr) return fail(ROPE_ERR_NULLPTR, why, "block_table is NULL");
        p.pages = k_cache->pages;
        p.page_size = k_cache->page_size;
        p.table_pages = table_pages;
    } else {
        p.page_size = 1;
    }
    p.table = block_table;
    p.table_stride = B > 1 ? table_stride : 0;
    p.lengths = lengths;
    p.counts = counts;
    // lengths are 32-bit numbers, so no sequence has 2^31 tokens or more
    p.most = p.table_pages > INT32_MAX / p.page_size ? INT32_MAX : p.table_pages * p.page_size;
    p.parts = attn_parts(B, p.heads, S * p.rep, p.most);
    const int64_t need = attn_workspace_bytes(B, S, q->N, p.heads, out->D);
    if (need > 0) {
        if (workspace == nullptr) return fail(ROPE_ERR_NULLPTR, why, "workspace is NULL");
        if (reinterpret_cast<uintptr_t>(workspace) % 16 != 0)
            return fail(ROPE_ERR_INVALID, why, "workspace must be 16-byte aligned");
        if (workspace_bytes < need) return fail(ROPE_ERR_INVALID, why, "workspace too small");
        p.part = static_cast<float*>(workspace);
    }
    *plan = p;
    return ROPE_OK;
}

}  // namespace rope
