// Argument checking of the cache entry points (see rope_cache_plan.hpp).
#include "rope_cache_plan.hpp"

#include <algorithm>
#include <limits>

namespace rope {

namespace {

constexpr int64_t kI64Max = std::numeric_limits<int64_t>::max();

rope_status_t fail(rope_status_t st, std::string* why, const std::string& msg)
{
    if (why) *why = msg;
    return st;
}

// Sum of (count - 1) * stride over dimensions plus `last`, or -1 past 64 bits.
int64_t extent(const int64_t counts[], const int64_t strides[], int n, int64_t last)
{
    int64_t sum = last;
    for (int i = 0; i < n; ++i) {
        if (counts[i] <= 1) continue;
        int64_t part;
        if (__builtin_mul_overflow(counts[i] - 1, strides[i], &part) || __builtin_add_overflow(sum, part, &sum))
            return -1;
    }
    return sum;
}

// Whether no two index triples reach a common element of rows of `width`:
// by rising stride, each dimension steps past everything the smaller ones
// cover. (Sufficient, and met by every slice or permutation of a tensor.)
bool disjoint_rows(const int64_t counts[3], const int64_t strides[3], int64_t width)
{
    int64_t c[3], s[3];
    int n = 0;
    for (int i = 0; i < 3; ++i)
        if (counts[i] > 1) {
            c[n] = counts[i];
            s[n++] = strides[i];
        }
    for (int i = 0; i < n; ++i)
        for (int j = i + 1; j < n; ++j)
            if (s[j] < s[i]) {
                std::swap(s[i], s[j]);
                std::swap(c[i], c[j]);
            }
    int64_t covered = width;
    for (int i = 0; i < n; ++i) {
        if (s[i] < covered) return false;
        covered += (c[i] - 1) * s[i];   // bounded by extent(), checked first
    }
    return true;
}

rope_status_t check_rows(const char* name, const rope_rows_t& r, int64_t B, int64_t S, int esize, bool written,
                         RowsPlan* p, std::string* why)
{
    for (int k = 0; k < 3; ++k)
        if (r.strides[k] < 0) return fail(ROPE_ERR_INVALID, why, std::string(name) + ": negative stride");
    const int64_t counts[3] = {B, S, r.N};
    const int64_t ext = extent(counts, r.strides, 3, r.D);
    if (ext < 0 || ext > kI64Max / esize)
        return fail(ROPE_ERR_INVALID, why, std::string(name) + ": strides overflow 64-bit offsets");
    if (written && !disjoint_rows(counts, r.strides, r.D))
        return fail(ROPE_ERR_INVALID, why, std::string(name) + ": its rows overlap each other");
    p->data = static_cast<char*>(r.data);
    p->N = r.N;
    p->D = r.D;
    p->sb = B > 1 ? r.strides[0] : 0;
    p->ss = S > 1 ? r.strides[1] : 0;
    p->sn = r.N > 1 ? r.strides[2] : 0;
    return ROPE_OK;
}

// A cache's own fields; `written`: its rows must not overlap.
rope_status_t check_cache(const char* name, const rope_cache_t& c, rope_dtype_t dtype, bool written, CachePlan* p,
                          std::string* why)
{
    const auto bad = [&](const std::string& msg) { return fail(ROPE_ERR_INVALID, why, std::string(name) + ": " + msg); };
    if (c.format < ROPE_CACHE_F32 || c.format > ROPE_CACHE_INT4) return bad("unknown format");
    p->quantised = c.format >= ROPE_CACHE_E4M3;
    if (!p->quantised && c.format != (int)dtype) return bad("its storage type must be that of the rows");
    if (c.pages < 0 || c.page_size < 0 || c.heads < 0 || c.dim < 0) return bad("negative dimension");
    if (c.dim % 2 != 0 || c.dim > ROPE_D_LIMIT) return bad("dim must be even and at most 1024");
    if (c.page_size > 0 && c.pages > kI64Max / c.page_size) return bad("too many slots");
    const int64_t counts[3] = {c.pages, c.page_size, c.heads};
    const int64_t width = cache_row_bytes(c.format, c.dim);
    const int es = p->quantised ? 1 : element_size(c.format);
    for (int k = 0; k < 3; ++k) {
        if (c.strides[k] < 0) return bad("negative stride");
        if (c.strides[k] % es != 0) return bad("a stride is not a whole number of elements");
        p->st[k] = counts[k] > 1 ? c.strides[k] : 0;
    }
    if (extent(counts, c.strides, 3, width) < 0) return bad("strides overflow 64-bit offsets");
    if (written && !disjoint_rows(counts, c.strides, width)) return bad("its rows overlap each other");
    if (p->quantised) {
        if (c.group < 2 || c.group % 2 != 0 || c.dim % c.group != 0) return bad("group must be even and divide dim");
        const int64_t groups = c.dim / c.group;
        for (int k = 0; k < 3; ++k) {
            if (c.scale_strides[k] < 0) return bad("negative scale stride");
            p->sc[k] = counts[k] > 1 ? c.scale_strides[k] : 0;
        }
        const int64_t ext = extent(counts, c.scale_strides, 3, groups);
        if (ext < 0 || ext > kI64Max / 4) return bad("scale strides overflow 64-bit offsets");
        if (written && !disjoint_rows(counts, c.scale_strides, groups)) return bad("its scales overlap each other");
    }
    p->data = static_cast<char*>(c.data);
    p->scales = c.scales;
    p->format = c.format;
    p->group = p->quantised ? c.group : c.dim;
    return ROPE_OK;
}

rope_status_t check_pointers(const char* name, const CachePlan& c, std::string* why)
{
    if (c.data == nullptr) return fail(ROPE_ERR_NULLPTR, why, std::string(name) + ": data is NULL");
    if (c.quantised && c.scales == nullptr) return fail(ROPE_ERR_NULLPTR, why, std::string(name) + ": scales is NULL");
    const uintptr_t es = c.quantised ? 1 : (uintptr_t)element_size(c.format);
    if (reinterpret_cast<uintptr_t>(c.data) % es != 0 || reinterpret_cast<uintptr_t>(c.scales) % 4 != 0)
        return fail(ROPE_ERR_INVALID, why, std::string(name) + ": data or scales not aligned to their elements");
    return ROPE_OK;
}

rope_status_t check_data(const char* name, const RowsPlan& r, int esize, std::string* why)
{
    if (r.data == nullptr) return fail(ROPE_ERR_NULLPTR, why, std::string(name) + ": data is NULL");
    if (reinterpret_cast<uintptr_t>(r.data) % (uintptr_t)esize != 0)
        return fail(ROPE_ERR_INVALID, why, std::string(name) + ": data not aligned to its elements");
    return ROPE_OK;
}

}  // namespace

rope_status_t make_cache_write_plan(int64_t B, int64_t S, rope_dtype_t dtype, const rope_rows_t* q,
                                    const rope_rows_t* k, const rope_rows_t* v, const rope_cache_t* k_cache,
                                    const rope_cache_t* v_cache, const int64_t* slots,
                                    const int64_t slots_strides[2], const Positions& in, rope_dtype_t table_dtype,
                                    int64_t mode, const int64_t partial_slice[2], bool rotate_k, CacheWritePlan* plan,
                                    std::string* why)
{
    CacheWritePlan p;
    if (k == nullptr || k_cache == nullptr) return fail(ROPE_ERR_NULLPTR, why, "k or k_cache is NULL");
    if ((v == nullptr) != (v_cache == nullptr))
        return fail(ROPE_ERR_NULLPTR, why, "v and v_cache must both be given or both be NULL");
    rope_status_t st = make_plan_scalars(B, S, k->N, k->D, dtype, table_dtype, mode, partial_slice, &p.rope, why);
    if (st != ROPE_OK) return st;
    const int es = p.rope.esize;
    if ((st = check_cache("k_cache", *k_cache, dtype, true, &p.kc, why)) != ROPE_OK) return st;
    if (k->N != k_cache->heads || k->D != k_cache->dim)
        return fail(ROPE_ERR_INVALID, why, "k: its heads and lanes must be the cache's");
    if ((st = check_rows("k", *k, B, S, es, false, &p.k, why)) != ROPE_OK) return st;
    p.pages = k_cache->pages;
    p.page_size = k_cache->page_size;
    if (v != nullptr) {
        if ((st = check_cache("v_cache", *v_cache, dtype, true, &p.vc, why)) != ROPE_OK) return st;
        if (v->N != v_cache->heads || v->D != v_cache->dim)
            return fail(ROPE_ERR_INVALID, why, "v: its heads and lanes must be the cache's");
        if (v->N < 0 || v->D < 0) return fail(ROPE_ERR_INVALID, why, "v: negative dimension");
        if (v_cache->pages != p.pages || v_cache->page_size != p.page_size)
            return fail(ROPE_ERR_INVALID, why, "v_cache: its pages must be k_cache's");
        if ((st = check_rows("v", *v, B, S, es, false, &p.v, why)) != ROPE_OK) return st;
        if (v->D == 0) p.v.N = 0;
    }
    if (q != nullptr) {
        if (q->N < 0) return fail(ROPE_ERR_INVALID, why, "q: negative dimension");
        if (q->D != k->D) return fail(ROPE_ERR_INVALID, why, "q: its lanes must be k's");
        if ((st = check_rows("q", *q, B, S, es, true, &p.q, why)) != ROPE_OK) return st;
    }
    if (p.rope.L == 0 || q == nullptr) p.q.N = 0;   // nothing to rotate in q
    if (p.k.D == 0) p.k.N = 0;
    p.B = B;
    p.S = S;
    int64_t tokens, rows;
    if (__builtin_mul_overflow(B, S, &tokens) || __builtin_add_overflow(p.q.N, p.k.N, &rows) ||
        __builtin_add_overflow(rows, p.v.N, &rows) || __builtin_mul_overflow(rows, tokens, &rows))
        return fail(ROPE_ERR_INVALID, why, "more rows than 64-bit offsets can address");
    if (rows == 0) {
        p.noop = true;
        *plan = p;
        return ROPE_OK;
    }
    if (rows >= (1ll << 31)) return fail(ROPE_ERR_UNSUPPORTED, why, "2^31 rows of q, k and v or more");
    if (p.k.N > 0) {
        if ((st = check_data("k", p.k, es, why)) != ROPE_OK) return st;
    }
    if (p.v.N > 0 && (st = check_data("v", p.v, es, why)) != ROPE_OK) return st;
    if (p.q.N > 0 && (st = check_data("q", p.q, es, why)) != ROPE_OK) return st;
    if (p.k.N > 0 || p.v.N > 0) {
        if (slots == nullptr || slots_strides == nullptr)
            return fail(ROPE_ERR_NULLPTR, why, "slots or slots_strides is NULL");
        if (slots_strides[0] < 0 || slots_strides[1] < 0)
            return fail(ROPE_ERR_INVALID, why, "slots: negative stride");
        const int64_t counts[2] = {B, S};
        const int64_t ext = extent(counts, slots_strides, 2, 1);
        if (ext < 0 || ext > kI64Max / 8) return fail(ROPE_ERR_INVALID, why, "slots: strides overflow 64-bit offsets");
        p.slots = slots;
        p.slot_sb = B > 1 ? slots_strides[0] : 0;
        p.slot_ss = S > 1 ? slots_strides[1] : 0;
        // a cache without slots takes no token: its pointers are not looked at
        if (p.pages > 0 && p.page_size > 0) {
            if (p.k.N > 0 && (st = check_pointers("k_cache", p.kc, why)) != ROPE_OK) return st;
            if (p.v.N > 0 && (st = check_pointers("v_cache", p.vc, why)) != ROPE_OK) return st;
        }
    }
    p.rotate_q = p.q.N > 0;
    p.rotate_k = rotate_k && p.k.N > 0 && p.rope.L > 0;
    if (p.rotate_q || p.rotate_k) {
        if ((st = check_positions(B, S, p.rope.L, in, &p.rope, why)) != ROPE_OK) return st;
    }
    *plan = p;
    return ROPE_OK;
}

rope_status_t make_cache_read_plan(int64_t B, int64_t S, rope_dtype_t dtype, const rope_rows_t* out,
                                   const rope_cache_t* cache, const int32_t* block_table, int64_t table_pages,
                                   int64_t table_stride, const int32_t* lengths, const int32_t* starts,
                                   const Positions& in, rope_dtype_t table_dtype, int64_t mode,
                                   const int64_t partial_slice[2], CacheReadPlan* plan, std::string* why)
{
    CacheReadPlan p;
    if (out == nullptr || cache == nullptr) return fail(ROPE_ERR_NULLPTR, why, "out or cache is NULL");
    rope_status_t st = make_plan_scalars(B, S, out->N, out->D, dtype, table_dtype, mode, partial_slice, &p.rope, why);
    if (st != ROPE_OK) return st;
    const int es = p.rope.esize;
    if ((st = check_cache("cache", *cache, dtype, false, &p.c, why)) != ROPE_OK) return st;
    if (out->N != cache->heads || out->D != cache->dim)
        return fail(ROPE_ERR_INVALID, why, "out: its heads and lanes must be the cache's");
    if ((st = check_rows("out", *out, B, S, es, true, &p.out, why)) != ROPE_OK) return st;
    if (table_pages < 0 || table_stride < 0) return fail(ROPE_ERR_INVALID, why, "block_table: negative size or stride");
    const int64_t counts[2] = {B, table_pages}, steps[2] = {table_stride, 1};
    const int64_t ext = extent(counts, steps, 2, 1);
    if (ext < 0 || ext > kI64Max / 4) return fail(ROPE_ERR_INVALID, why, "block_table: stride overflows 64-bit offsets");
    p.B = B;
    p.S = S;
    p.pages = cache->pages;
    p.page_size = cache->page_size;
    int64_t tokens, rows;
    if (__builtin_mul_overflow(B, S, &tokens) || __builtin_mul_overflow(tokens, out->N, &rows))
        return fail(ROPE_ERR_INVALID, why, "more rows than 64-bit offsets can address");
    if (rows == 0 || out->D == 0 || p.pages == 0 || p.page_size == 0 || table_pages == 0) {
        p.noop = true;
        *plan = p;
        return ROPE_OK;
    }
    if (rows >= (1ll << 31)) return fail(ROPE_ERR_UNSUPPORTED, why, "2^31 rows or more");
    if ((st = check_data("out", p.out, es, why)) != ROPE_OK) return st;
    if ((st = check_pointers("cache", p.c, why)) != ROPE_OK) return st;
    if (block_table == nullptr || lengths == nullptr)
        return fail(ROPE_ERR_NULLPTR, why, "block_table or lengths is NULL");
    p.table = block_table;
    p.table_pages = table_pages;
    p.table_stride = B > 1 ? table_stride : 0;
    p.lengths = lengths;
    p.starts = starts;
    p.rotate = in.data != nullptr && p.rope.L > 0;
    if (p.rotate && (st = check_positions(B, S, p.rope.L, in, &p.rope, why)) != ROPE_OK) return st;
    *plan = p;
    return ROPE_OK;
}

}  // namespace rope
