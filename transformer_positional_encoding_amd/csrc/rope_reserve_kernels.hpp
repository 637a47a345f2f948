// rope_reserve_kernels.hpp -- pages of a paged cache given to growing sequences
// and taken back from shrinking ones, with the slots and positions of the new
// tokens. Included by rope_reserve.hip.
//
// Everything follows from two running sums over the sequences: of the pages
// that each gives back and of those that each needs. Page number i of those
// given back goes to place c + i of the list of free pages (c: its count), page
// number k of those needed comes from place c' - 1 - k (c': with the pages
// given back). A thread takes one of these numbers and finds its sequence by
// bisection, so that a sequence of many pages costs no more steps than many of
// a few. It is all latency; the steps are ordered so that two suffice: what
// reads the lengths, the old table and the count of free pages (reserve_take),
// and what replaces them (reserve_finish). Calls of few tokens run both in one
// block (a launch less); others in two launches of many blocks, each block
// with the running sums for itself. 256 sequences of a token each 7.7 us, 48
// prompts of 4096 tokens 12.7 (7.6 and 5.1).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rope_fastdiv.hpp"

namespace rope {
namespace {

struct ReserveArgs {
    int32_t* table;
    int64_t cols, table_stride;
    int32_t* lengths;
    const int32_t* counts;
    int32_t* free_pages;
    int32_t* free_count;
    int32_t capacity;          // of free_pages
    uint32_t B, S;
    uint64_t tokens;           // B * S, below 2^31
    int64_t* slots;
    int64_t* positions;
    int32_t* granted;
    FastDiv page_div, s_div;
};

constexpr int kReserveThreads = 1024;
constexpr int32_t kReserveMost = 0x7fffffff;

__device__ __forceinline__ int32_t sat_add(int32_t a, int32_t b)     // of numbers that are not negative
{
    const uint32_t s = (uint32_t)a + (uint32_t)b;
    return s > (uint32_t)kReserveMost ? kReserveMost : (int32_t)s;
}

// Pages of n tokens.
__device__ __forceinline__ int32_t pages_of(const ReserveArgs& a, int32_t n)
{
    return n <= 0 ? 0 : (int32_t)fast_div((uint32_t)n - 1, a.page_div) + 1;
}

// What a sequence asks for: its tokens now and those it keeps, the pages it
// gives back or needs; whether it can grow at all.
struct Ask {
    int32_t old, kept, gives, needs;
    bool fits;
};

__device__ __forceinline__ Ask ask_of(const ReserveArgs& a, uint32_t b)
{
    Ask k;
    k.old = a.lengths[b];
    const int32_t n = a.counts[b];
    const int64_t room = (int64_t)a.page_div.d * a.cols;
    const bool sound = k.old >= 0 && k.old <= room;
    k.kept = k.old;
    k.gives = k.needs = 0;
    k.fits = false;
    if (!sound) return k;
    if (n < 0) {
        const int64_t left = (int64_t)k.old + n;
        k.kept = left > 0 ? (int32_t)left : 0;
        k.gives = pages_of(a, k.old) - pages_of(a, k.kept);
    } else if (n > 0) {
        const int64_t grown = (int64_t)k.old + n;
        k.fits = (uint32_t)n <= a.S && grown <= room && grown <= kReserveMost;
        if (k.fits) k.needs = pages_of(a, (int32_t)grown) - pages_of(a, k.old);
    }
    return k;
}

// Running sums (the last included) of both kinds of pages, in LDS.
__device__ __forceinline__ void reserve_sums(const ReserveArgs& a, int32_t* gives, int32_t* needs)
{
    __shared__ int32_t wave_sums[2][kReserveThreads / 64];
    const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const uint32_t per = (a.B + kReserveThreads - 1) / kReserveThreads;
    const uint32_t b0 = min(a.B, t * per), b1 = min(a.B, b0 + per);
    int32_t g = 0, n = 0;
    for (uint32_t b = b0; b < b1; ++b) {
        const Ask k = ask_of(a, b);
        gives[b] = g = sat_add(g, k.gives);
        needs[b] = n = sat_add(n, k.needs);
    }
    int32_t sg = g, sn = n;                  // over the threads of a wave, then over waves
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t og = __shfl_up(sg, d), on = __shfl_up(sn, d);
        if (lane >= (uint32_t)d) {
            sg = sat_add(sg, og);
            sn = sat_add(sn, on);
        }
    }
    if (lane == 63) {
        wave_sums[0][wave] = sg;
        wave_sums[1][wave] = sn;
    }
    int32_t bg = __shfl_up(sg, 1), bn = __shfl_up(sn, 1);
    if (lane == 0) bg = bn = 0;
    __syncthreads();
    for (uint32_t w = 0; w < wave; ++w) {
        bg = sat_add(bg, wave_sums[0][w]);
        bn = sat_add(bn, wave_sums[1][w]);
    }
    for (uint32_t b = b0; b < b1; ++b) {
        gives[b] = sat_add(gives[b], bg);
        needs[b] = sat_add(needs[b], bn);
    }
    __syncthreads();
}

// The first of n rising sums that is larger than v (n if none).
__device__ __forceinline__ uint32_t first_above(const int32_t* sums, uint32_t n, int32_t v)
{
    uint32_t lo = 0, hi = n;
    while (lo < hi) {
        const uint32_t mid = (lo + hi) / 2;
        if (sums[mid] > v) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// Page number i of those given back.
__device__ __forceinline__ int32_t given_page(const ReserveArgs& a, const int32_t* gives, int32_t i)
{
    const uint32_t b = first_above(gives, a.B, i);
    const Ask k = ask_of(a, b);
    const int32_t before = gives[b] - k.gives;
    return a.table[b * a.table_stride + pages_of(a, k.kept) + (i - before)];
}

__device__ __forceinline__ void reserve_take(const ReserveArgs& a, int32_t* lds, uint32_t block, uint32_t blocks)
{
    int32_t *gives = lds, *needs = lds + a.B;
    reserve_sums(a, gives, needs);
    const uint64_t first = (uint64_t)block * kReserveThreads + threadIdx.x, step = (uint64_t)blocks * kReserveThreads;
    const int32_t count = min(max(*a.free_count, 0), a.capacity);
    // pages given back (no more than the list holds), then those needed
    const int32_t back = min(gives[a.B - 1], a.capacity - count);
    const int32_t have = count + back;
    const uint32_t refused = first_above(needs, a.B, have);
    const int32_t taken = refused == 0 ? 0 : needs[refused - 1];
    for (uint64_t i = first; i < (uint64_t)back; i += step) a.free_pages[count + i] = given_page(a, gives, (int32_t)i);
    for (uint64_t i = first; i < (uint64_t)taken; i += step) {
        const int32_t k = (int32_t)i;
        const uint32_t b = first_above(needs, a.B, k);
        const Ask ask = ask_of(a, b);
        const int32_t place = have - 1 - k;
        const int32_t page = place < count ? a.free_pages[place] : given_page(a, gives, place - count);
        a.table[b * a.table_stride + pages_of(a, ask.old) + (k - (needs[b] - ask.needs))] = page;
    }
    for (uint64_t b = first; b < a.B; b += step) {
        const Ask k = ask_of(a, (uint32_t)b);
        const bool given = k.fits && (k.needs == 0 || needs[b] <= have);
        a.granted[b] = given ? a.counts[b] : k.kept - k.old;
    }
    for (uint64_t i = first; i < a.tokens; i += step) {
        const uint32_t b = fast_div((uint32_t)i, a.s_div), s = (uint32_t)i - b * a.S;
        a.positions[i] = (int64_t)max(ask_of(a, b).kept, 0) + s;
    }
}

__device__ __forceinline__ void reserve_finish(const ReserveArgs& a, uint32_t block, uint32_t blocks)
{
    __shared__ int32_t totals[2];
    const uint64_t first = (uint64_t)block * kReserveThreads + threadIdx.x, step = (uint64_t)blocks * kReserveThreads;
    for (uint64_t i = first; i < a.tokens; i += step) {
        const uint32_t b = fast_div((uint32_t)i, a.s_div), s = (uint32_t)i - b * a.S;
        int64_t slot = -1;
        if ((int64_t)s < (int64_t)a.granted[b]) {
            const uint32_t at = (uint32_t)a.positions[i];
            const uint32_t col = fast_div(at, a.page_div);
            const int32_t page = a.table[b * a.table_stride + col];
            if (page >= 0) slot = (int64_t)page * a.page_div.d + (at - col * a.page_div.d);
        }
        a.slots[i] = slot;
    }
    // columns that were given back, a wave a sequence
    const uint32_t lane = threadIdx.x & 63;
    for (uint64_t b = first >> 6; b < a.B; b += step >> 6) {
        const int32_t g = a.granted[b];
        if (g >= 0) continue;
        const int32_t kept = (int32_t)a.positions[b * a.S];
        const int32_t c0 = pages_of(a, kept), c1 = pages_of(a, kept - g);
        for (int32_t c = c0 + (int32_t)lane; c < c1; c += 64) a.table[b * a.table_stride + c] = -1;
    }
    // the lengths; the free pages that are left
    if (threadIdx.x == 0) totals[0] = totals[1] = 0;
    __syncthreads();
    int32_t gave = 0, took = 0;
    if (block == 0) {
        for (uint32_t b = threadIdx.x; b < a.B; b += kReserveThreads) {
            const int32_t g = a.granted[b], from = (int32_t)a.positions[(uint64_t)b * a.S];
            if (g > 0) took += pages_of(a, from + g) - pages_of(a, from);
            if (g < 0) gave = sat_add(gave, pages_of(a, from - g) - pages_of(a, from));
            if (g != 0) a.lengths[b] = g > 0 ? from + g : from;
        }
        if (took != 0) atomicAdd(&totals[0], took);       // no more than the list holds
        if (gave != 0) {                                  // may pass 32 bits where a table is not sound
            int32_t seen = totals[1], was;
            do {
                was = seen;
                seen = atomicCAS(&totals[1], was, sat_add(was, gave));
            } while (seen != was);
        }
    }
    __syncthreads();
    if (block == 0 && threadIdx.x == 0) {
        const int32_t count = min(max(*a.free_count, 0), a.capacity);
        *a.free_count = count + min(totals[1], a.capacity - count) - totals[0];
    }
}

__global__ void __launch_bounds__(kReserveThreads) rope_reserve_block_kernel(ReserveArgs a)
{
    extern __shared__ int32_t sums_lds[];
    reserve_take(a, sums_lds, 0, 1);
    __syncthreads();
    reserve_finish(a, 0, 1);
}

__global__ void __launch_bounds__(kReserveThreads) rope_reserve_take_kernel(ReserveArgs a)
{
    extern __shared__ int32_t sums_lds[];
    reserve_take(a, sums_lds, blockIdx.x, gridDim.x);
}

__global__ void __launch_bounds__(kReserveThreads) rope_reserve_finish_kernel(ReserveArgs a)
{
    reserve_finish(a, blockIdx.x, gridDim.x);
}

}  // namespace
}  // namespace rope
