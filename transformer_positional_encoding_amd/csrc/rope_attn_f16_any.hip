// The matrix-core attention kernels for f16 queries, pages of any size.
#include "rope_attn_select.hpp"

namespace rope {

const void* attn_kernel_f16_any(int lanes, int scales, AttnRowsOf rows)
{
    return attn_kernel<ROPE_DTYPE_F16, false>(lanes, scales, rows);
}

}  // namespace rope
