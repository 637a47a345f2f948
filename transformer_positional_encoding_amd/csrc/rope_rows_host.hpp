// What the host code of the calls on strided rows and caches shares: kernel
// arguments from checked plans, and whether rows fall into 8-lane chunks.
#pragma once

#include <algorithm>
#include <string>

#include "rope_cache_kernels.hpp"
#include "rope_cache_plan.hpp"
#include "rope_host.hpp"

namespace rope {
namespace {

inline Rows rows_of(const RowsPlan& p) { return Rows{p.data, p.sb, p.ss, p.sn}; }

inline CacheRef cache_of(const CachePlan& p)
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

inline Turn turn_of(const Plan& p)
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

// Whether 8-lane chunks of these rows are 16-byte aligned.
inline bool rows_in_chunks(const RowsPlan& r, int esize)
{
    const int64_t per = 16 / esize;
    return r.N == 0 || (r.D % 8 == 0 && aligned16(r.data) && r.sb % per == 0 && r.ss % per == 0 && r.sn % per == 0);
}

// Whether the slice is whole chunks whose partners are in the chunk or whole
// chunks away.
inline bool turn_in_chunks(const Plan& p)
{
    return p.start % 8 == 0 && p.L % 8 == 0 && (p.half == 1 || p.half % 8 == 0);
}

inline bool power_of_two(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }

inline uint32_t log2_of(uint32_t v)
{
    uint32_t s = 0;
    while ((1u << s) < v) ++s;
    return s;
}

inline rope_status_t launched(hipError_t err)
{
    if (err != hipSuccess) return set_error(ROPE_ERR_RUNTIME, std::string("kernel launch: ") + hipGetErrorString(err));
    return ROPE_OK;
}

}  // namespace
}  // namespace rope
