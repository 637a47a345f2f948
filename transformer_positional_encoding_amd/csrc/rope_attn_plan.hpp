// Host-side checks of attention over a paged cache (rope_cache_attention).
// Pure C++ (no HIP), so they run without a GPU.
#pragma once

#include "rope_cache_plan.hpp"

namespace rope {

// Parts of all sequences, by heads and tiles of rows, that fill the card (waves:
// two a SIMD, where blocks of four heads are two a compute unit. 64 sequences of
// up to 8192 tokens, one new one: 132 us by 1024, 100 by 2048, 104 by 4096; 16
// of 5 new ones 81, 72 and 93); most that one sequence's tokens are divided
// into; most sequences that are.
constexpr int64_t kAttnBlocks = 2048;
constexpr int64_t kAttnMaxParts = 512;
constexpr int64_t kAttnMaxSplit = 1024;

struct AttnPlan {
    Plan rope;                     // dimensions and storage type
    int64_t B = 0, S = 0;
    RowsPlan q, out;
    CachePlan kc, vc;
    int64_t heads = 0;             // of the caches
    int64_t rep = 0;               // rows of q for each of them
    int64_t pages = 0, page_size = 0;
    int64_t most = 0;              // tokens that a block table holds, below 2^31
    const int32_t* table = nullptr;
    int64_t table_pages = 0, table_stride = 0;
    const int32_t* lengths = nullptr;
    const int32_t* counts = nullptr;
    double scale = 0;
    bool causal = false;
    float* part = nullptr;         // partial results
    int64_t parts = 0;             // that the sequences' tokens are divided into; B: not divided
    bool noop = false;
};

// Parts for B sequences of `heads` cached heads and `rows` rows of each over up
// to `tokens` cached tokens: as many as fill the card, if that is a quarter more
// than sequences.
int64_t attn_parts(int64_t B, int64_t heads, int64_t rows, int64_t tokens);

// Bytes of workspace for any number of tokens; 0 when nothing is computed or
// the arguments are out of range.
int64_t attn_workspace_bytes(int64_t B, int64_t S, int64_t q_heads, int64_t heads, int64_t Dv);

rope_status_t make_attn_plan(int64_t B, int64_t S, rope_dtype_t dtype, const rope_rows_t* out, const rope_rows_t* q,
                             const rope_cache_t* k_cache, const rope_cache_t* v_cache, const int32_t* block_table,
                             int64_t table_pages, int64_t table_stride, const int32_t* lengths, const int32_t* counts,
                             double scale, bool causal, void* workspace, int64_t workspace_bytes, AttnPlan* plan,
                             std::string* why);

}  // namespace rope
