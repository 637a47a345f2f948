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
    t.ax.last = p.naxes > 0 ? (uint32_t)(p.naxes - 1) : 0;
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
    a.n_div = make_fastdiv(a.N);
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

hipError_t launch_write(const CacheWritePlan& p, hipStream_t s)
{
    CacheWriteArgs a = write_args(p);
    void* args[] = {&a};
    return hipLaunchKernel(by_types<WriteGeneral>(p.rope.dtype, kernel_format(p.kc)), dim3(general_grid(a.rows)),
                           dim3(kGenThreads), args, 0, s);
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
    rope::CacheReadArgs a = rope::read_args(p);
    void* args[] = {&a};
    return rope::launched(hipLaunchKernel(rope::by_types<rope::ReadGeneral>(p.rope.dtype, rope::kernel_format(p.c)),
                                          dim3(rope::general_grid(a.rows)), dim3(rope::kGenThreads), args, 0,
                                          static_cast<hipStream_t>(stream)));
}

}  // extern "C"
