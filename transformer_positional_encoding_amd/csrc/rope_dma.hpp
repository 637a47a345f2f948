// rope_dma.hpp -- loads from global memory straight to LDS, and the wait for
// them. Included by the kernels that stage tiles this way.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rope {
namespace {

// One direct global-to-LDS load of 16 bytes per lane from base + voff (base
// the same for the whole wave, voff lane l's byte offset): lane l's bytes go
// to LDS byte address lds_base + 16*l (lds_base the same for the whole wave).
// (A load to LDS may not follow a write of m0 at once.)
__device__ __forceinline__ void lds_dma16(const void* base, uint32_t voff, uint32_t lds_base)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds_base), "v"(voff), "s"(base) : "memory");
}

// The same from an address of each lane's own.
__device__ __forceinline__ void lds_dma16_far(const void* p, uint32_t lds_base)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds_base), "v"(p) : "memory");
}

// s_waitcnt vmcnt(N) with lgkmcnt and expcnt left free (gfx9 encoding:
// vmcnt bits [3:0] and [15:14], expcnt [6:4], lgkmcnt [11:8]).
template <int N>
__device__ __forceinline__ void wait_vm()
{
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

}  // namespace
}  // namespace rope
