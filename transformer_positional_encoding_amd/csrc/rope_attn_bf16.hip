// The matrix-core attention kernels for bf16 queries, pages of whole 16 tokens.
#include "rope_attn_select.hpp"

namespace rope {

const void* attn_kernel_bf16(int lanes, int scales, AttnRowsOf rows)
{
    return attn_kernel<ROPE_DTYPE_BF16, true>(lanes, scales, rows);
}

}  // namespace rope
