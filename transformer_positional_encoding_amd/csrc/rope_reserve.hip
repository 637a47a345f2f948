// Pages, slots and positions of a step's new tokens.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <limits>
#include <string>

#include "rope_host.hpp"
#include "rope_reserve_kernels.hpp"

namespace rope {
namespace {

// Tokens up to which one block does all of a call: a launch less. (In a graph,
// one block and two launches: 256 tokens 8.2 us and 9.5, 4096 of 256 sequences
// 13.6 and 10.8, 8192 of 4 7.6 and 6.2, 16384 of 256 25.9 and 10.9.)
constexpr uint64_t kReserveOneBlock = kReserveThreads;

hipError_t launch_reserve(ReserveArgs a, hipStream_t s)
{
    const size_t lds = 2 * (size_t)a.B * sizeof(int32_t);
    void* args[] = {&a};
    if (a.tokens <= kReserveOneBlock)
        return hipLaunchKernel(reinterpret_cast<const void*>(&rope_reserve_block_kernel), dim3(1), dim3(kReserveThreads), args,
                               lds, s);
    const uint32_t blocks = (uint32_t)std::min<uint64_t>(256, (a.tokens + kReserveThreads - 1) / kReserveThreads);
    hipError_t err = hipLaunchKernel(reinterpret_cast<const void*>(&rope_reserve_take_kernel), dim3(blocks),
                                     dim3(kReserveThreads), args, lds, s);
    if (err != hipSuccess) return err;
    return hipLaunchKernel(reinterpret_cast<const void*>(&rope_reserve_finish_kernel), dim3(blocks), dim3(kReserveThreads),
                           args, 0, s);
}

rope_status_t reserve_args(int64_t B, int64_t S, int32_t* block_table, int64_t table_pages, int64_t table_stride,
                           int32_t* lengths, const int32_t* counts, int32_t* free_pages, int64_t capacity,
                           int32_t* free_count, int64_t page_size, int64_t* slots, int64_t* positions, int32_t* granted,
                           ReserveArgs* a, std::string* why)
{
    const auto bad = [&](rope_status_t st, const char* msg) {
        *why = msg;
        return st;
    };
    constexpr int64_t kMax32 = std::numeric_limits<int32_t>::max();
    if (B < 0 || S < 1) return bad(ROPE_ERR_INVALID, "B must not be negative and S at least 1");
    if (table_pages < 0 || table_stride < 0) return bad(ROPE_ERR_INVALID, "block_table: negative size or stride");
    if (B > 1 && table_stride < table_pages) return bad(ROPE_ERR_INVALID, "block_table: its rows overlap each other");
    if (page_size < 1) return bad(ROPE_ERR_INVALID, "page_size must be at least 1");
    if (capacity < 0) return bad(ROPE_ERR_INVALID, "free_pages: negative capacity");
    if (B == 0) return ROPE_OK;
    if (B > ROPE_RESERVE_MAX) return bad(ROPE_ERR_UNSUPPORTED, "more than ROPE_RESERVE_MAX sequences");
    if (S > kMax32 / B || page_size > kMax32 || capacity > kMax32 || table_pages > kMax32)
        return bad(ROPE_ERR_UNSUPPORTED, "B * S, page_size, capacity or table_pages of 2^31 or more");
    if (table_stride > std::numeric_limits<int64_t>::max() / 4 / B)
        return bad(ROPE_ERR_INVALID, "block_table: stride overflows 64-bit offsets");
    if (lengths == nullptr || counts == nullptr || free_count == nullptr || slots == nullptr || positions == nullptr ||
        granted == nullptr || (block_table == nullptr && table_pages > 0) || (free_pages == nullptr && capacity > 0))
        return bad(ROPE_ERR_NULLPTR, "block_table, lengths, counts, free_pages, free_count, slots, positions or granted is NULL");
    const uintptr_t small = reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(lengths) |
                            reinterpret_cast<uintptr_t>(counts) | reinterpret_cast<uintptr_t>(free_pages) |
                            reinterpret_cast<uintptr_t>(free_count) | reinterpret_cast<uintptr_t>(granted);
    const uintptr_t wide = reinterpret_cast<uintptr_t>(slots) | reinterpret_cast<uintptr_t>(positions);
    if (small % 4 != 0 || wide % 8 != 0) return bad(ROPE_ERR_INVALID, "an array is not aligned to its elements");
    a->table = block_table;
    a->cols = table_pages;
    a->table_stride = B > 1 ? table_stride : 0;
    a->lengths = lengths;
    a->counts = counts;
    a->free_pages = free_pages;
    a->free_count = free_count;
    a->capacity = (int32_t)capacity;
    a->B = (uint32_t)B;
    a->S = (uint32_t)S;
    a->tokens = (uint64_t)(B * S);
    a->slots = slots;
    a->positions = positions;
    a->granted = granted;
    a->page_div = make_fastdiv((uint32_t)page_size);
    a->s_div = make_fastdiv((uint32_t)S);
    return ROPE_OK;
}

}  // namespace
}  // namespace rope

extern "C" rope_status_t rope_cache_reserve(
    int64_t B, int64_t S, int32_t* block_table, int64_t table_pages, int64_t table_stride, int32_t* lengths,
    const int32_t* counts, int32_t* free_pages, int64_t free_capacity, int32_t* free_count, int64_t page_size,
    int64_t* slots, int64_t* positions, int32_t* granted, void* stream)
{
    rope::ReserveArgs a{};
    std::string why;
    rope_status_t st = rope::reserve_args(B, S, block_table, table_pages, table_stride, lengths, counts, free_pages,
                                          free_capacity, free_count, page_size, slots, positions, granted, &a, &why);
    if (st != ROPE_OK) return rope::set_error(st, why);
    if (B == 0) return ROPE_OK;
    const hipError_t err = rope::launch_reserve(a, static_cast<hipStream_t>(stream));
    if (err != hipSuccess) return rope::set_error(ROPE_ERR_RUNTIME, std::string("kernel launch: ") + hipGetErrorString(err));
    return ROPE_OK;
}
