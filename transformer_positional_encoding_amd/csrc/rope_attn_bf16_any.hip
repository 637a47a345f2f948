// The matrix-core attention kernels for bf16 queries, pages of any size.
#include "rope_attn_select.hpp"

namespace rope {

const void* attn_kernel_bf16_any(int lanes, int scales, AttnRowsOf rows)
{
    return attn_kernel<ROPE_DTYPE_BF16, false>(lanes, scales, rows);
}

}  // namespace rope
