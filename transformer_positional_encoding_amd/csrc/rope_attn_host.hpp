// What the attention's launch and its kernels' translation units share.
#pragma once

namespace rope {

// Scales of a cached row: one of K and one of V; K's by 32-lane steps (also
// where rows are short of the kernel's lanes, or not aligned for one load), V's
// one; both by 32-lane segments; by halves of those, K's or V's or both (one tile
// of rows).
constexpr int kAttnRowScales = 0;
constexpr int kAttnKSegments = 1;
constexpr int kAttnSegments = 2;
constexpr int kAttnKHalves = 3;
constexpr int kAttnVHalves = 4;
constexpr int kAttnHalves = 5;

// Query rows of a cached head that a kernel takes: 16 or 32 a wave, by waves on
// their own, or 32 a wave, 128 a block, whose waves share their tiles' numbers
// (16 and 64 with scales of halves), or 16 or 32 a wave of one of four heads that
// a block loads together.
enum class AttnRowsOf { kOneTile, kTwoTiles, kShared, kFourHeads, kFourHeadsTwoTiles };

// The kernel for rows of up to `lanes` lanes (64, 128; 256: kOneTile only;
// kFourHeads: pages of whole 16 tokens only).
// _any: for pages of any size, the others for pages of whole 16 tokens less
// than 2^26 bytes apart.
const void* attn_kernel_bf16(int lanes, int scales, AttnRowsOf rows);
const void* attn_kernel_f16(int lanes, int scales, AttnRowsOf rows);
const void* attn_kernel_bf16_any(int lanes, int scales, AttnRowsOf rows);
const void* attn_kernel_f16_any(int lanes, int scales, AttnRowsOf rows);

}  // namespace rope
