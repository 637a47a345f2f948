// Host-side checks of the cache entry points (rope_cache_write,
// rope_cache_read). Pure C++ (no HIP), so they run without a GPU.
#pragma once

#include "rope_plan.hpp"

namespace rope {

// Rows of q, k, v or out, normalised: strides of size-1 dimensions are 0.
struct RowsPlan {
    char* data = nullptr;
    int64_t N = 0, D = 0;
    int64_t sb = 0, ss = 0, sn = 0;   // elements
};

struct CachePlan {
    char* data = nullptr;
    float* scales = nullptr;
    int format = 0;
    bool quantised = false;
    int64_t group = 0;
    int64_t st[3] = {0, 0, 0};    // bytes: page, slot, head
    int64_t sc[3] = {0, 0, 0};    // floats
};

struct CacheWritePlan {
    Plan rope;                    // k's geometry, slice, mode, positions
    int64_t B = 0, S = 0;
    RowsPlan q, k, v;             // q.N or v.N 0 when there is none (or q needs no rotation)
    CachePlan kc, vc;
    int64_t pages = 0, page_size = 0;
    const int64_t* slots = nullptr;
    int64_t slot_sb = 0, slot_ss = 0;
    bool rotate_q = false, rotate_k = false;
    bool noop = false;
};

struct CacheReadPlan {
    Plan rope;
    int64_t B = 0, S = 0;
    RowsPlan out;
    CachePlan c;
    int64_t pages = 0, page_size = 0;
    const int32_t* table = nullptr;
    int64_t table_pages = 0, table_stride = 0;
    const int32_t* lengths = nullptr;
    const int32_t* starts = nullptr;
    bool rotate = false;
    bool noop = false;
};

// The codes of a row take this many bytes.
inline int64_t cache_row_bytes(int format, int64_t dim)
{
    switch (format) {
    case ROPE_CACHE_F32: return 4 * dim;
    case ROPE_CACHE_F16:
    case ROPE_CACHE_BF16: return 2 * dim;
    case ROPE_CACHE_INT4: return dim / 2;
    default: return dim;
    }
}

rope_status_t make_cache_write_plan(int64_t B, int64_t S, rope_dtype_t dtype, const rope_rows_t* q,
                                    const rope_rows_t* k, const rope_rows_t* v, const rope_cache_t* k_cache,
                                    const rope_cache_t* v_cache, const int64_t* slots,
                                    const int64_t slots_strides[2], const Positions& in, rope_dtype_t table_dtype,
                                    int64_t mode, const int64_t partial_slice[2], bool rotate_k, CacheWritePlan* plan,
                                    std::string* why);

rope_status_t make_cache_read_plan(int64_t B, int64_t S, rope_dtype_t dtype, const rope_rows_t* out,
                                   const rope_cache_t* cache, const int32_t* block_table, int64_t table_pages,
                                   int64_t table_stride, const int32_t* lengths, const int32_t* starts,
                                   const Positions& in, rope_dtype_t table_dtype, int64_t mode,
                                   const int64_t partial_slice[2], CacheReadPlan* plan, std::string* why);

}  // namespace rope
