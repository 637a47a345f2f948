// The cache entry points: rotated keys (and values, and queries beside them)
// to a paged, quantised cache in one launch, and cached tokens read back.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <string>

#include "rope_cache_kernels.hpp"
#include "rope_cache_plan.hpp"
#include "rope_host.hpp"

namespace rope {
namespace {

Rows rows_of(const RowsPlan& p) { return Rows{p.data, p.sb, p.ss, p.sn}; }

CacheRef cache_of(const CachePlan& p)
{
    CacheRef c{};
    c.data = p.data;
    c.scales = p.scales;
    for (int k = 0; k < 3; ++k) {
        c.st[k] = p.st[k];
        c.sc[k] = p.sc[k];
    }
    c.group = (uint32_t)std::max<int64_t>(1, p.group);
    return c;
}

Turn turn_of(const Plan& p)
{
    Turn t{};
    t.pos = p.pos;
    t.inv_freq = p.inv_freq;
    t.sb = p.pos_sb;
    t.ss = p.pos_ss;
    t.ax.sa = p.pos_sa;
    t.ax.nwords = p.naxes > 1 ? (uint32_t)((p.L / 2 + 15) / 16) : 0;
    std::copy(std::begin(p.axis_words), std::end(p.axis_words), t.ax.words);
    t.tdt = p.tdtype;
    t.start = (uint32_t)p.start;
    t.L = (uint32_t)p.L;
    t.half = (uint32_t)std::max<int64_t>(1, p.half);
    t.pairs = (uint32_t)(p.L / 2);
    t.half_div = make_fastdiv(t.half);
    return t;
}

int kernel_format(const CachePlan& c) { return c.quantised ? c.format : kFmtSame; }

uint32_t general_grid(uint64_t rows)
{
    return (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>(rows, kMaxGridItems / kGenThreads));
}

CacheWriteArgs write_args(const CacheWritePlan& p)
{
    CacheWriteArgs a{};
    a.q = rows_of(p.q);
    a.k = rows_of(p.k);
    a.v = rows_of(p.v);
    a.kc = cache_of(p.kc);
    a.vc = cache_of(p.vc);
    a.Nq = (uint32_t)p.q.N;
    a.Nk = (uint32_t)p.k.N;
    a.Nv = (uint32_t)p.v.N;
    a.Dk = (uint32_t)p.rope.D;
    a.Dv = (uint32_t)p.v.D;
    a.tokens = (uint32_t)(p.B * p.S);
    a.S = (uint32_t)p.S;
    a.rows = (uint64_t)a.tokens * (a.Nq + a.Nk + a.Nv);
    a.slots = p.slots;
    a.slot_sb = p.slot_sb;
    a.slot_ss = p.slot_ss;
    a.page_size = std::max<int64_t>(1, p.page_size);
    a.nslots = p.pages * p.page_size;
    a.rotate_k = p.rotate_k ? 1 : 0;
    a.turn = turn_of(p.rope);
    a.s_div = make_fastdiv(a.S);
    a.row_div = make_fastdiv(a.Nq + a.Nk + a.Nv);
    return a;
}

CacheReadArgs read_args(const CacheReadPlan& p)
{
    CacheReadArgs a{};
    a.out = rows_of(p.out);
    a.c = cache_of(p.c);
    a.N = (uint32_t)p.out.N;
    a.D = (uint32_t)p.rope.D;
    a.S = (uint32_t)p.S;
    a.rows = (uint64_t)p.B * (uint64_t)p.S * (uint64_t)p.out.N;
    a.table = p.table;
    a.table_pages = p.table_pages;
    a.table_stride = p.table_stride;
    a.lengths = p.lengths;
    a.starts = p.starts;
    a.pages = p.pages;
    a.page_size = p.page_size;
    a.rotate = p.rotate ? 1 : 0;
    a.turn = turn_of(p.rope);
    a.s_div = make_fastdiv(a.S);
    return a;
}

// A kernel for a storage type and a cache format.
template <template <int, int> class K>
const void* by_types(int dtype, int fmt)
{
    const auto f = [&](auto dt) -> const void* {
        constexpr int DT = decltype(dt)::value;
        switch (fmt) {
        case kFmtE4M3: return K<DT, kFmtE4M3>::ptr();
        case kFmtInt8: return K<DT, kFmtInt8>::ptr();
        case kFmtInt4: return K<DT, kFmtInt4>::ptr();
        default: return K<DT, kFmtSame>::ptr();
        }
    };
    switch (dtype) {
    case ROPE_DTYPE_F32: return f(std::integral_constant<int, ROPE_DTYPE_F32>{});
    case ROPE_DTYPE_F16: return f(std::integral_constant<int, ROPE_DTYPE_F16>{});
    default: return f(std::integral_constant<int, ROPE_DTYPE_BF16>{});
    }
}

template <int DT, int FMT>
struct WriteGeneral {
    static const void* ptr() { return reinterpret_cast<const void*>(&rope_cache_write_general_kernel<DT, FMT>); }
};
template <int DT, int FMT>
struct ReadGeneral {
    static const void* ptr() { return reinterpret_cast<const void*>(&rope_cache_read_general_kernel<DT, FMT>); }
};

template <int C, bool PAR>
struct WriteVec {
    template <int DT, int FMT>
    struct K {
        static const void* ptr() { return reinterpret_cast<const void*>(&rope_cache_write_kernel<DT, FMT, C, PAR>); }
    };
};

template <bool PAR>
const void* write_kernel(int C, int dtype, int fmt)
{
    switch (C) {
    case 1: return by_types<WriteVec<1, PAR>::template K>(dtype, fmt);
    case 2: return by_types<WriteVec<2, PAR>::template K>(dtype, fmt);
    default: return by_types<WriteVec<3, PAR>::template K>(dtype, fmt);
    }
}

template <int DT, int FMT>
struct ReadVec {
    static const void* ptr() { return reinterpret_cast<const void*>(&rope_cache_read_kernel<DT, FMT, false>); }
};
template <int DT, int FMT>
struct ReadVecTurn {
    static const void* ptr() { return reinterpret_cast<const void*>(&rope_cache_read_kernel<DT, FMT, true>); }
};
template <int DT, int FMT>
struct ReadWave {
    static const void* ptr() { return reinterpret_cast<const void*>(&rope_cache_read_wave_kernel<DT, FMT, false>); }
};
template <int DT, int FMT>
struct ReadWaveTurn {
    static const void* ptr() { return reinterpret_cast<const void*>(&rope_cache_read_wave_kernel<DT, FMT, true>); }
};

// Whether 8-lane chunks of these rows are 16-byte aligned.
bool rows_in_chunks(const RowsPlan& r, int esize)
{
    const int64_t per = 16 / esize;
    return r.N == 0 || (r.D % 8 == 0 && aligned16(r.data) && r.sb % per == 0 && r.ss % per == 0 && r.sn % per == 0);
}

// Whether the codes of 8 lanes are aligned to their size.
bool cache_in_chunks(const CachePlan& c)
{
    const uintptr_t bytes = !c.quantised ? 16 : c.format == ROPE_CACHE_INT4 ? 4 : 8;
    if (reinterpret_cast<uintptr_t>(c.data) % bytes != 0) return false;
    for (int k = 0; k < 3; ++k)
        if (c.st[k] % (int64_t)bytes != 0) return false;
    return true;
}

// Whether the slice is whole chunks whose partners are in the chunk or whole
// chunks away.
bool turn_in_chunks(const Plan& p)
{
    return p.start % 8 == 0 && p.L % 8 == 0 && (p.half == 1 || p.half % 8 == 0);
}

bool power_of_two(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }

uint32_t log2_of(uint32_t v)
{
    uint32_t s = 0;
    while ((1u << s) < v) ++s;
    return s;
}

// Chunks per scale for the write kernel: 0 for one scale a row; -1 if the
// kernel does not take the group.
int group_chunks(const CachePlan& c, int64_t D)
{
    if (!c.quantised || c.group == D) return 0;
    return c.group % 8 == 0 && power_of_two(c.group / 8) && c.group / 8 <= 64 ? (int)(c.group / 8) : -1;
}

// The vector write kernel's arguments and shape; false if a row or a group
// is not in whole chunks.
bool write_vec_args(const CacheWritePlan& p, CacheWriteVecArgs* a, int* C, uint32_t* grid, size_t* lds)
{
    const int es = p.rope.esize;
    if (!rows_in_chunks(p.q, es) || !rows_in_chunks(p.k, es) || !rows_in_chunks(p.v, es)) return false;
    if ((p.k.N > 0 && !cache_in_chunks(p.kc)) || (p.v.N > 0 && !cache_in_chunks(p.vc))) return false;
    const bool turning = p.rotate_q || p.rotate_k;
    if (turning && !turn_in_chunks(p.rope)) return false;
    const int gk = p.k.N > 0 ? group_chunks(p.kc, p.k.D) : 0, gv = p.v.N > 0 ? group_chunks(p.vc, p.v.D) : 0;
    if (gk < 0 || gv < 0) return false;
    // Threads per row and chunks per thread: the fewest idle lanes; among
    // those the most chunks per thread that leave a row 8 threads (128 bytes
    // of 16-bit lanes a load).
    const uint32_t chunks = (uint32_t)std::max(p.q.N + p.k.N > 0 ? p.rope.D : 0, p.v.N > 0 ? p.v.D : 0) / 8;
    uint32_t best = ~0u;
    for (uint32_t c = 1; c <= 3; ++c) {
        const uint32_t T = 1u << log2_of(std::max<uint32_t>((chunks + c - 1) / c, (uint32_t)std::max(std::max(gk, gv), 1)));
        if (T > 64) continue;
        const uint32_t cost = 2 * T * c + (T < 8 ? 1 : 0);
        if (cost < best || (cost == best && T >= 8)) {
            best = cost;
            a->T = T;
            *C = (int)c;
        }
    }
    if (best == ~0u) return false;
    a->rows_per_block = kVecThreads / a->T;
    a->t_div = make_fastdiv(a->T);
    if (!turning) a->turn.L = a->turn.pairs = 0;
    a->own_partner = *C == 2 && p.rope.start == 0 && p.rope.half == 8 * (int64_t)a->T && p.rope.L == 2 * p.rope.half;
    a->gvk = (uint32_t)gk;
    a->gvv = (uint32_t)gv;
    a->small_slots = a->nslots < (1ll << 31);
    a->page_div = make_fastdiv(a->small_slots ? (uint32_t)std::max<int64_t>(1, std::min<int64_t>(a->page_size, INT32_MAX)) : 1);
    a->pairs_div = make_fastdiv(std::max<uint32_t>(1, a->turn.pairs));
    a->nq_div = make_fastdiv(std::max<uint32_t>(1, a->Nq));
    a->nk_div = make_fastdiv(std::max<uint32_t>(1, a->Nk));
    a->nv_div = make_fastdiv(std::max<uint32_t>(1, a->Nv));
    const auto blocks = [&](uint32_t N) { return ((uint64_t)a->tokens * N + a->rows_per_block - 1) / a->rows_per_block; };
    // tokens that a block's rows of a kind can span
    const auto spans = [&](uint32_t N) { return N == 0 ? 0 : (a->rows_per_block + N - 2) / N + 1; };
    const uint64_t all = blocks(a->Nq) + blocks(a->Nk) + blocks(a->Nv);
    if (all > kMaxGridItems / kVecThreads) return false;
    a->blocks_q = (uint32_t)blocks(a->Nq);
    a->blocks_k = (uint32_t)blocks(a->Nk);
    *grid = (uint32_t)all;
    a->lds_floats = std::max(spans(a->Nq), a->rotate_k ? spans(a->Nk) : 0) * a->turn.pairs;
    *lds = 2 * (size_t)a->lds_floats * sizeof(float);
    return *lds <= 64 * 1024;
}

hipError_t launch_write(const CacheWritePlan& p, hipStream_t s)
{
    const int fmt = kernel_format(p.k.N > 0 ? p.kc : p.v.N > 0 ? p.vc : p.kc);
    CacheWriteVecArgs v{};
    static_cast<CacheWriteArgs&>(v) = write_args(p);
    int C = 1;
    uint32_t grid = 0;
    size_t lds = 0;
    if (write_vec_args(p, &v, &C, &grid, &lds)) {
        void* args[] = {&v};
        const bool par = v.turn.L > 0 && v.turn.half != 1;
        const void* fn = par ? write_kernel<true>(C, p.rope.dtype, fmt) : write_kernel<false>(C, p.rope.dtype, fmt);
        return hipLaunchKernel(fn, dim3(grid), dim3(kVecThreads), args, lds, s);
    }
    CacheWriteArgs a = write_args(p);
    void* args[] = {&a};
    return hipLaunchKernel(by_types<WriteGeneral>(p.rope.dtype, fmt), dim3(general_grid(a.rows)), dim3(kGenThreads),
                           args, 0, s);
}

// Whether a wave takes a token of so many chunks, with so many pairs to turn
// (measured figures at the kernels): where the token is one full pass of the
// wave, unless its lanes idle over the cos and sin of 32 pairs or fewer, or
// enough passes that the last one's open lanes weigh little.
bool read_by_wave(uint32_t chunks, uint32_t pairs)
{
    if (chunks == 64) return pairs == 0 || pairs > 32;
    return chunks > (pairs == 0 ? 96u : 127u);
}

hipError_t launch_read(const CacheReadPlan& p, hipStream_t s)
{
    CacheReadVecArgs a{};
    static_cast<CacheReadArgs&>(a) = read_args(p);
    const int fmt = kernel_format(p.c);
    const int64_t groups = p.rope.D / p.c.group;
    a.chunks = (uint32_t)(p.rope.D / 8);
    const uint64_t items = a.rows * a.chunks;
    const bool vec = p.rope.D % 8 == 0 && rows_in_chunks(p.out, p.rope.esize) && cache_in_chunks(p.c) &&
                     (!p.rotate || turn_in_chunks(p.rope)) && (groups == 1 || (p.c.group % 8 == 0 && power_of_two(p.c.group / 8))) &&
                     items < (1ull << 31);
    if (vec) {
        a.token_chunks = a.N * a.chunks;
        a.tokens = (uint32_t)(p.B * p.S);
        a.group_shift = groups == 1 ? 31 : log2_of((uint32_t)(p.c.group / 8));
        a.small_tokens = p.table_pages <= (int64_t)INT32_MAX / p.page_size;
        a.chunk_div = make_fastdiv(a.chunks);
        a.token_div = make_fastdiv(a.token_chunks);
        a.page_div = make_fastdiv(a.small_tokens ? (uint32_t)p.page_size : 1);
        a.pairs_div = make_fastdiv(std::max<uint32_t>(1, a.turn.pairs));
        void* args[] = {&a};
        const int dt = p.rope.dtype;
        const bool wave = read_by_wave(a.token_chunks, p.rotate ? a.turn.pairs : 0);
        const void* fn = wave ? (p.rotate ? by_types<ReadWaveTurn>(dt, fmt) : by_types<ReadWave>(dt, fmt))
                              : (p.rotate ? by_types<ReadVecTurn>(dt, fmt) : by_types<ReadVec>(dt, fmt));
        // (a wave's token has 64 chunks or more, so its grid fits as the block's)
        const uint32_t block = kReadChunks * kVecThreads;
        const uint32_t grid = wave ? (a.tokens + 3) / 4 : (uint32_t)((items + block - 1) / block);
        // tokens that a block's chunks can span: at most 4 pairs for each of its
        // chunks and of two tokens of 127, 25 KB of cos and sin
        const size_t spans = (block + a.token_chunks - 2) / a.token_chunks + 1;
        const size_t lds = !wave && p.rotate ? 2 * spans * a.turn.pairs * sizeof(float) : 0;
        return hipLaunchKernel(fn, dim3(grid), dim3(kVecThreads), args, lds, s);
    }
    CacheReadArgs g = a;
    void* args[] = {&g};
    const uint64_t blocks = std::min<uint64_t>((uint64_t)p.B * (uint64_t)p.S, kMaxGridItems / kGenReadThreads);
    return hipLaunchKernel(by_types<ReadGeneral>(p.rope.dtype, fmt), dim3((uint32_t)blocks), dim3(kGenReadThreads), args,
                           0, s);
}

rope_status_t launched(hipError_t err)
{
    if (err != hipSuccess) return set_error(ROPE_ERR_RUNTIME, std::string("kernel launch: ") + hipGetErrorString(err));
    return ROPE_OK;
}

}  // namespace
}  // namespace rope

extern "C" {

rope_status_t rope_cache_write(
    int64_t B, int64_t S, rope_dtype_t dtype, const rope_rows_t* q, const rope_rows_t* k, const rope_rows_t* v,
    const rope_cache_t* k_cache, const rope_cache_t* v_cache, const int64_t* slots, const int64_t slots_strides[2],
    const int64_t* positions, const int64_t positions_shape[3], const int64_t positions_strides[3],
    const double* inv_freq, const int32_t* pair_axes, rope_dtype_t table_dtype, int64_t mode,
    const int64_t partial_slice[2], int32_t rotate_k, void* stream)
{
    rope::CacheWritePlan p;
    std::string why;
    const rope::Positions in{positions, positions_shape, positions_strides, inv_freq, true, pair_axes, true};
    rope_status_t st = rope::make_cache_write_plan(B, S, dtype, q, k, v, k_cache, v_cache, slots, slots_strides, in,
                                                   table_dtype, mode, partial_slice, rotate_k != 0, &p, &why);
    if (st != ROPE_OK) return rope::set_error(st, why);
    if (p.noop) return ROPE_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (p.v.N > 0 && rope::kernel_format(p.vc) != rope::kernel_format(p.kc)) {
        // v in another format than k: a launch each, v's rows in k's place
        rope::CacheWritePlan kp = p, vp = p;
        kp.v.N = 0;
        vp.q.N = vp.k.N = 0;
        vp.rotate_q = vp.rotate_k = false;
        vp.kc = p.vc;
        hipError_t err = kp.q.N + kp.k.N > 0 ? rope::launch_write(kp, s) : hipSuccess;
        if (err == hipSuccess) err = rope::launch_write(vp, s);
        return rope::launched(err);
    }
    return rope::launched(rope::launch_write(p, s));
}

rope_status_t rope_cache_read(
    int64_t B, int64_t S, rope_dtype_t dtype, const rope_rows_t* out, const rope_cache_t* cache,
    const int32_t* block_table, int64_t table_pages, int64_t table_stride, const int32_t* lengths,
    const int32_t* starts, const int64_t* positions, const int64_t positions_shape[3],
    const int64_t positions_strides[3], const double* inv_freq, const int32_t* pair_axes, rope_dtype_t table_dtype,
    int64_t mode, const int64_t partial_slice[2], void* stream)
{
    rope::CacheReadPlan p;
    std::string why;
    const rope::Positions in{positions, positions_shape, positions_strides, inv_freq, true, pair_axes, true};
    rope_status_t st = rope::make_cache_read_plan(B, S, dtype, out, cache, block_table, table_pages, table_stride,
                                                  lengths, starts, in, table_dtype, mode, partial_slice, &p, &why);
    if (st != ROPE_OK) return rope::set_error(st, why);
    if (p.noop) return ROPE_OK;
    return rope::launched(rope::launch_read(p, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
