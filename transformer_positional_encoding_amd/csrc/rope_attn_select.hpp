// The matrix-core attention kernels by what their template arguments stand for.
// Included by the rope_attn_*.hip files of a type each, which compile side by
// side.
#pragma once

#include "rope_attn_mfma_kernels.hpp"
#include "rope_attn_host.hpp"

namespace rope {
namespace {

template <int DT, int DP, bool P16, int NT>
const void* attn_by_scales(int scales)
{
    switch (scales) {
    case kAttnRowScales: return reinterpret_cast<const void*>(&rope_attn_mfma_kernel<DT, DP, DP, false, false, P16, NT>);
    case kAttnKSegments: return reinterpret_cast<const void*>(&rope_attn_mfma_kernel<DT, DP, DP, true, false, P16, NT>);
    default: return reinterpret_cast<const void*>(&rope_attn_mfma_kernel<DT, DP, DP, true, true, P16, NT>);
    }
}

template <int DT, bool P16>
const void* attn_kernel(int lanes, int scales, int tiles)
{
    switch (lanes) {
    case 64: return tiles == 1 ? attn_by_scales<DT, 64, P16, 1>(scales) : attn_by_scales<DT, 64, P16, 2>(scales);
    case 128: return tiles == 1 ? attn_by_scales<DT, 128, P16, 1>(scales) : attn_by_scales<DT, 128, P16, 2>(scales);
    default: return attn_by_scales<DT, 256, P16, 1>(scales);
    }
}

}  // namespace
}  // namespace rope
