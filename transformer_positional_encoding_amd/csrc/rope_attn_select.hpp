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
    case kAttnRowScales: return reinterpret_cast<const void*>(&rope_attn_mfma_kernel<DT, DP, DP, 0, 0, P16, NT>);
    case kAttnKSegments: return reinterpret_cast<const void*>(&rope_attn_mfma_kernel<DT, DP, DP, 1, 0, P16, NT>);
    case kAttnKHalves: return reinterpret_cast<const void*>(&rope_attn_mfma_kernel<DT, DP, DP, kHalves, 0, P16, 1>);
    case kAttnVHalves: return reinterpret_cast<const void*>(&rope_attn_mfma_kernel<DT, DP, DP, 1, kHalves, P16, 1>);
    case kAttnHalves: return reinterpret_cast<const void*>(&rope_attn_mfma_kernel<DT, DP, DP, kHalves, kHalves, P16, 1>);
    default: return reinterpret_cast<const void*>(&rope_attn_mfma_kernel<DT, DP, DP, 1, 1, P16, NT>);
    }
}

template <int DT, int DP, bool P16>
const void* attn_shared(int scales)
{
    switch (scales) {
    case kAttnRowScales: return reinterpret_cast<const void*>(&rope_attn_shared_kernel<DT, DP, 0, 0, P16, 2>);
    case kAttnKSegments: return reinterpret_cast<const void*>(&rope_attn_shared_kernel<DT, DP, 1, 0, P16, 2>);
    case kAttnSegments: return reinterpret_cast<const void*>(&rope_attn_shared_kernel<DT, DP, 1, 1, P16, 2>);
    case kAttnKHalves: return reinterpret_cast<const void*>(&rope_attn_shared_kernel<DT, DP, kHalves, 0, P16, 1>);
    case kAttnVHalves: return reinterpret_cast<const void*>(&rope_attn_shared_kernel<DT, DP, 1, kHalves, P16, 1>);
    default: return reinterpret_cast<const void*>(&rope_attn_shared_kernel<DT, DP, kHalves, kHalves, P16, 1>);
    }
}

template <int DT, int DP, int NT>
const void* attn_heads(int scales)
{
    switch (scales) {
    case kAttnRowScales: return reinterpret_cast<const void*>(&rope_attn_heads_kernel<DT, DP, 0, 0, NT>);
    case kAttnKSegments: return reinterpret_cast<const void*>(&rope_attn_heads_kernel<DT, DP, 1, 0, NT>);
    case kAttnKHalves: return reinterpret_cast<const void*>(&rope_attn_heads_kernel<DT, DP, kHalves, 0, 1>);
    case kAttnVHalves: return reinterpret_cast<const void*>(&rope_attn_heads_kernel<DT, DP, 1, kHalves, 1>);
    case kAttnHalves: return reinterpret_cast<const void*>(&rope_attn_heads_kernel<DT, DP, kHalves, kHalves, 1>);
    default: return reinterpret_cast<const void*>(&rope_attn_heads_kernel<DT, DP, 1, 1, NT>);
    }
}

template <int DT, int DP, bool P16>
const void* attn_by_rows(int scales, AttnRowsOf rows)
{
    switch (rows) {
    case AttnRowsOf::kOneTile: return attn_by_scales<DT, DP, P16, 1>(scales);
    case AttnRowsOf::kTwoTiles: return attn_by_scales<DT, DP, P16, 2>(scales);
    case AttnRowsOf::kFourHeads:
        if constexpr (P16) return attn_heads<DT, DP, 1>(scales);
        return nullptr;
    case AttnRowsOf::kFourHeadsTwoTiles:
        if constexpr (P16) return attn_heads<DT, DP, 2>(scales);
        return nullptr;
    default: return attn_shared<DT, DP, P16>(scales);
    }
}

template <int DT, bool P16>
const void* attn_kernel(int lanes, int scales, AttnRowsOf rows)
{
    switch (lanes) {
    case 64: return attn_by_rows<DT, 64, P16>(scales, rows);
    case 128: return attn_by_rows<DT, 128, P16>(scales, rows);
    default: return attn_by_scales<DT, 256, P16, 1>(scales);
    }
}

}  // namespace
}  // namespace rope
