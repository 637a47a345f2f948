// rope_attn_kernels.hpp -- attention of new tokens over a paged cache held in 4
// bits. Included by rope_attn.hip, next to the host code that launches them.
//
// Mathematics. A sequence's query rows q (the new tokens by the heads that share
// a cached head) and cached tokens t, with k_t and v_t codes times the scales of
// their groups of lanes:
//   x_t = scale q.k_t,  m = max x_t,  l = sum exp(x_t - m),  o = sum exp(x_t - m) v_t / l
// over the tokens that a row sees, in one pass with the running m, l and o. A
// part of a sequence's tokens leaves m, l and sum exp(x_t - m) v_t; parts are
// joined in order by a second kernel.
#pragma once

#include <type_traits>

#include "rope_attn_plan.hpp"
#include "rope_cache_kernels.hpp"

namespace rope {
namespace {

constexpr float kAttnNone = -__builtin_inff();   // the maximum of nothing

struct AttnArgs {
    Rows q, out;
    CacheRef kc, vc;
    uint32_t D, Dv, S, Hq, heads, rep;
    uint32_t rows;             // of a cached head: S * rep; row r is token r / rep, head r % rep of the group
    uint32_t tiles;            // of rows
    uint32_t B, parts;         // of all sequences' tokens
    bool split;                // parts > B: results are joined
    uint32_t most_parts;       // of one sequence
    uint32_t unit;             // tokens that a part is whole multiples of
    const int32_t* table;
    int64_t table_stride;
    const int32_t* lengths;
    const int32_t* counts;
    int64_t pages;
    uint32_t page_limit;       // pages, as far as 32-bit numbers name them
    int32_t most;              // tokens that a block table holds
    float scale2;              // scale * log2(e)
    int32_t causal;
    int32_t words;             // general kernel: K's codes by whole aligned words of 8
    float* part;               // per part, token and head: Dv sums; then m and l of all
    uint32_t part_rows;        // of a part: S * Hq
    FastDiv rep_div, heads_div, tiles_div, page_div;
};

// A block's place: cached head (or group of heads), tile of rows, part, the
// first changing fastest: heads lie beside each other in memory, and what blocks
// read at the same time should too.
struct AttnAt {
    uint32_t part, tile, head, b;
    uint32_t first, end;       // the part's tokens, as many as there are
};

// A sequence: its cached tokens, its new ones, and the place of the first.
struct AttnSeq {
    int32_t tokens;            // that the block table holds
    int32_t count;             // rows that are computed
    int64_t first;             // query s stands at token first + s
};

__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs& a, uint32_t b)
{
    AttnSeq s;
    const int32_t length = a.lengths[b];
    const int32_t count = a.counts != nullptr ? a.counts[b] : (int32_t)a.S;
    s.count = min(max(count, 0), (int32_t)a.S);
    s.first = (int64_t)length - s.count;
    s.tokens = min(max(length, 0), a.most);
    return s;
}

// Sums of the lanes up to each one, and the largest of all lanes.
__device__ __forceinline__ uint32_t lanes_up_to(uint32_t v)
{
    const auto from = [&](auto ctrl, auto rows) {
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
    };
    using All = std::integral_constant<int, 0xF>;
    v += from(std::integral_constant<int, 0x111>{}, All{});        // lanes of 16: 1, 2, 4, 8 before
    v += from(std::integral_constant<int, 0x112>{}, All{});
    v += from(std::integral_constant<int, 0x114>{}, All{});
    v += from(std::integral_constant<int, 0x118>{}, All{});
    v += from(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});
    v += from(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});
    return v;
}
__device__ __forceinline__ uint32_t lanes_sum(uint32_t v) { return __builtin_amdgcn_readlane((int)lanes_up_to(v), 63); }
__device__ __forceinline__ uint32_t lanes_max(uint32_t v)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d));
    return __builtin_amdgcn_readfirstlane((int)v);
}

// Sequences are split into parts of the same number of tokens, whatever each
// one's length, so that blocks end together: a.parts of them at most, which is
// all that the host can know. Every wave finds out for itself (and so do those that
// join), from the lengths: the smallest part, within 1/16, that makes no more.
// 16 sequences of up to 8000 tokens, 5 new ones each, 40 heads on 8: every one
// in as many parts as the others 90 us, so 72; 64 such 290 and 197. (What a
// sequence's sums are taken in parts of then depends on the batch's lengths.)
struct AttnShare {
    uint32_t b, first, n;      // a sequence, its first part and how many
    uint32_t per;              // units of a part
};
constexpr int kAttnBatch = kAttnMaxSplit / 64;

// Of the sequence that part `key` belongs to (b = a.B: of none), or of sequence
// `key` itself.
template <bool PART>
__device__ __forceinline__ AttnShare attn_share(const AttnArgs& a, uint32_t key)
{
    if (a.B == 1) {                                // (the same without the sums)
        const AttnSeq seq = attn_seq(a, 0);
        const uint32_t units = seq.count > 0 ? ((uint32_t)seq.tokens + a.unit - 1) / a.unit : 0, parts = min(a.parts, a.most_parts);
        const uint32_t per = max(1u, (units + parts - 1) / parts), n = (units + per - 1) / per;
        return AttnShare{PART && key >= n, 0, n, per};
    }
    const uint32_t lane = threadIdx.x & 63;
    uint32_t u[kAttnBatch], high = 0, low = 0, most = 0;
#pragma unroll
    for (int c = 0; c < kAttnBatch; ++c) {
        u[c] = 0;
        if (c * 64 >= a.B) continue;
        const uint32_t b = c * 64 + lane;
        if (b < a.B) {
            const AttnSeq seq = attn_seq(a, b);
            u[c] = seq.count > 0 ? ((uint32_t)seq.tokens + a.unit - 1) / a.unit : 0;
        }
        high += u[c] >> 10;
        low += u[c] & 1023;
        most = max(most, u[c]);
    }
    high = lanes_sum(high);
    low = lanes_sum(low);
    most = lanes_max(most);
    AttnShare s{a.B, 0, 0, 0};
    s.per = max(max(1u, (most + a.most_parts - 1) / a.most_parts),
                high / a.parts * 1024 + (high % a.parts * 1024 + low) / a.parts);
    for (;; s.per += max(1u, s.per / 16)) {        // (ends: one part each is B, of no more than a.parts)
        uint32_t n = 0;
#pragma unroll
        for (int c = 0; c < kAttnBatch; ++c)
            if (c * 64 < a.B) n += (u[c] + s.per - 1) / s.per;
        if (lanes_sum(n) <= a.parts) break;
    }
#pragma unroll
    for (int c = 0; c < kAttnBatch; ++c) {
        if (c * 64 >= a.B || s.b != a.B) continue;
        const uint32_t n = (u[c] + s.per - 1) / s.per, up_to = lanes_up_to(n);
        const uint64_t hit = PART ? __ballot(s.first + up_to > key) : key / 64 == (uint32_t)c ? 1ull << (key & 63) : 0;
        if (hit != 0) {
            const int at = __builtin_ctzll(hit);
            s.b = c * 64 + at;
            s.n = __builtin_amdgcn_readlane((int)n, at);
            s.first += __builtin_amdgcn_readlane((int)up_to, at) - s.n;
        } else {
            s.first += __builtin_amdgcn_readlane((int)up_to, 63);
        }
    }
    return s;
}

// False: nothing to do.
__device__ __forceinline__ bool attn_at(const AttnArgs& a, uint32_t block, AttnAt* p)
{
    const uint32_t i = fast_div(block, a.heads_div);
    p->head = block - i * a.heads_div.d;
    p->part = fast_div(i, a.tiles_div);
    p->tile = i - p->part * a.tiles;
    p->b = p->part;
    p->first = 0;
    p->end = UINT32_MAX;
    if (!a.split) return true;
    const AttnShare s = attn_share<true>(a, p->part);
    if (s.b == a.B) return false;
    p->b = s.b;
    // (tokens are fewer than 2^31)
    p->first = (uint32_t)min((uint64_t)INT32_MAX, (uint64_t)(p->part - s.first) * s.per * a.unit);
    p->end = (uint32_t)min((uint64_t)INT32_MAX, (uint64_t)(p->part - s.first + 1) * s.per * a.unit);
    return true;
}

// The tokens [*t0, *t1) of a part that are among the first n.
__device__ __forceinline__ void attn_part(const AttnAt& at, uint32_t n, uint32_t* t0, uint32_t* t1)
{
    *t0 = min(at.first, n);
    *t1 = min(at.end, n);
}

// The partial result of (part, token, head).
__device__ __forceinline__ uint64_t part_row(const AttnArgs& a, uint32_t part, uint32_t s, uint32_t h)
{
    return (uint64_t)part * a.part_rows + (uint64_t)s * a.Hq + h;
}

__device__ __forceinline__ float2* part_stats(const AttnArgs& a)
{
    return reinterpret_cast<float2*>(a.part + (uint64_t)a.parts * a.part_rows * a.Dv);
}

// How much a part counts whose maximum is m.
__device__ __forceinline__ float part_weight(float m, float most)
{
    return m == kAttnNone ? 0.0f : m == most ? 1.0f : exp2f(m - most);
}
__device__ __forceinline__ float one_over(float sum) { return sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum; }   // NaN stays

// a * b, 0 where a is 0: a scale that is infinite or NaN reaches only the rows
// that see its token. (Not right behind a transcendental or matrix instruction
// that makes an operand: nothing waits for those here.)
__device__ __forceinline__ float mul_or_0(float a, float b)
{
    float r;
    asm("v_mul_legacy_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}

// ---------------------------------------------------------------------------
// General kernel: any dimensions, groups, alignment and types, all in fp32. A
// block takes up to 4 rows that share a cached head, 256 tokens at a time: a
// thread a token's products with q (a word of 8 codes at a time where words are
// aligned and groups hold them whole), then a thread a byte of v's rows, two
// lanes, of every so many tokens. q and the weights stand in LDS with the four
// rows' values together. Bound by its instructions: 16 sequences of up to 8192
// tokens, 32 heads on 8 of 128 lanes, float32: 156 us (0.7 TB/s).
// ---------------------------------------------------------------------------
constexpr int kAttnGenThreads = 256;
constexpr int kAttnGenRows = 4;
constexpr int kAttnGenBytes = ROPE_D_LIMIT / 2 / kAttnGenThreads;      // of v's row, a thread, at most
constexpr int kAttnGenAhead = 4;                   // tokens whose loads go out together

// The code in bits 4 i to 4 i + 3.
__device__ __forceinline__ float code_of(uint32_t w, int i) { return (float)((int32_t)(w << (28 - 4 * i)) >> 28); }

template <int DT>
__global__ void __launch_bounds__(kAttnGenThreads) rope_attn_general_kernel(AttnArgs a)
{
    __shared__ float4 q[ROPE_D_LIMIT];
    __shared__ float4 p[kAttnGenThreads];
    __shared__ int64_t v_at[kAttnGenThreads], vs_at[kAttnGenThreads];
    __shared__ float red[kAttnGenRows][kAttnGenThreads / 64];
    const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6;
    AttnAt at;
    if (!attn_at(a, blockIdx.x, &at)) return;    // the same for the whole block
    const AttnSeq seq = attn_seq(a, at.b);
    const uint32_t r0 = at.tile * kAttnGenRows;
    const uint32_t live = min(a.rows, (uint32_t)seq.count * a.rep);
    if (r0 >= live) return;                      // the same for the whole block
    const uint32_t nr = min((uint32_t)kAttnGenRows, live - r0);
    for (uint32_t j = t; j < a.D; j += kAttnGenThreads) {
        float v[kAttnGenRows] = {};
#pragma unroll
        for (int r = 0; r < kAttnGenRows; ++r) {
            if (r >= (int)nr) continue;
            const uint32_t s = fast_div(r0 + r, a.rep_div), h = at.head * a.rep + (r0 + r - s * a.rep);
            v[r] = Store<DT>::load1(a.q.data, at.b * a.q.sb + s * a.q.ss + h * a.q.sn + j);
        }
        q[j] = make_float4(v[0], v[1], v[2], v[3]);
    }
    // this thread's bytes of v's rows, and its turn among the tokens
    const uint32_t v_bytes = a.Dv / 2;
    uint32_t cols = 1;
    while (cols < v_bytes && cols < (uint32_t)kAttnGenThreads) cols *= 2;
    const uint32_t strands = kAttnGenThreads / cols, strand = t / cols, col = t & (cols - 1);
    float m[kAttnGenRows], l[kAttnGenRows], o[kAttnGenBytes][2][kAttnGenRows];
    int64_t last[kAttnGenRows];                  // the last token that the row sees
#pragma unroll
    for (int r = 0; r < kAttnGenRows; ++r) {
        m[r] = kAttnNone;
        l[r] = 0.0f;
#pragma unroll
        for (int k = 0; k < kAttnGenBytes; ++k) o[k][0][r] = o[k][1][r] = 0.0f;
        last[r] = a.causal ? seq.first + fast_div(min(r0 + r, a.rows - 1), a.rep_div) : INT64_MAX;
    }
    uint32_t from, to;
    attn_part(at, (uint32_t)seq.tokens, &from, &to);
    const bool words = a.words != 0;
    __syncthreads();
    for (uint32_t base = from; base < to; base += kAttnGenThreads) {
        const uint32_t tok = base + t;
        int64_t page = -1, in_page = 0;
        if (tok < to) {
            const uint32_t c = fast_div(tok, a.page_div);
            page = a.table[at.b * a.table_stride + c];
            in_page = tok - c * a.page_div.d;
        }
        const bool there = page >= 0 && page < a.pages;
        float x[kAttnGenRows] = {};
        if (there) {
            const gchar* k = as_global(a.kc.data) + page * a.kc.st[0] + in_page * a.kc.st[1] + at.head * a.kc.st[2];
            const float* ks = a.kc.scales + page * a.kc.sc[0] + in_page * a.kc.sc[1] + at.head * a.kc.sc[2];
            for (uint32_t g = 0, j = 0; j < a.D; ++g) {
                float dot[kAttnGenRows] = {};
                const uint32_t end = j + a.kc.group;
                while (j < end) {
                    const int n = words ? 8 : 2;
                    const uint32_t w = words ? gload<uint32_t>(k + j / 2) : (uint32_t)gload<uint8_t>(k + j / 2);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (i >= n) break;
                        const float c = code_of(w, i);
                        const float4 v = q[j + i];
                        dot[0] = __builtin_fmaf(v.x, c, dot[0]);
                        dot[1] = __builtin_fmaf(v.y, c, dot[1]);
                        dot[2] = __builtin_fmaf(v.z, c, dot[2]);
                        dot[3] = __builtin_fmaf(v.w, c, dot[3]);
                    }
                    j += n;
                }
                const float scale = ks[g];
#pragma unroll
                for (int r = 0; r < kAttnGenRows; ++r) x[r] = __builtin_fmaf(dot[r], scale, x[r]);
            }
        }
        v_at[t] = there ? page * a.vc.st[0] + in_page * a.vc.st[1] + at.head * a.vc.st[2] : -1;
        vs_at[t] = page * a.vc.sc[0] + in_page * a.vc.sc[1] + at.head * a.vc.sc[2];
        // the tile's maxima
#pragma unroll
        for (int r = 0; r < kAttnGenRows; ++r) {
            x[r] = there && (int64_t)tok <= last[r] ? x[r] * a.scale2 : kAttnNone;
            float most = x[r];
            for (int d = 1; d < 64; d <<= 1) most = fmaxf(most, __shfl_xor(most, d));
            if (lane == 0) red[r][wave] = most;
        }
        __syncthreads();
        float e[kAttnGenRows];
#pragma unroll
        for (int r = 0; r < kAttnGenRows; ++r) {
            float most = m[r];
            for (int w = 0; w < kAttnGenThreads / 64; ++w) most = fmaxf(most, red[r][w]);
            const float keep = m[r] == most ? 1.0f : exp2f(m[r] - most);
            m[r] = most;
            const bool seen = there && (int64_t)tok <= last[r];
            e[r] = !seen ? 0.0f : exp2f(x[r] - most);
            l[r] = l[r] * keep + e[r];           // this thread's share
#pragma unroll
            for (int k = 0; k < kAttnGenBytes; ++k) {
                o[k][0][r] *= keep;
                o[k][1][r] *= keep;
            }
        }
        p[t] = make_float4(e[0], e[1], e[2], e[3]);
        __syncthreads();
        const uint32_t n = min((uint32_t)kAttnGenThreads, to - base);
#pragma unroll
        for (int k = 0; k < kAttnGenBytes; ++k) {
            const uint32_t byte = k * kAttnGenThreads + col;
            if (byte >= v_bytes) continue;
            const uint32_t g = 2 * byte / a.vc.group;              // (groups are even)
            for (uint32_t i = strand; i < n; i += strands * kAttnGenAhead) {
                uint32_t w[kAttnGenAhead];
                float scale[kAttnGenAhead];
#pragma unroll
                for (int u = 0; u < kAttnGenAhead; ++u) {
                    const uint32_t one = i + u * strands;
                    w[u] = 0;
                    scale[u] = 0.0f;
                    if (one >= n || v_at[one] < 0) continue;
                    w[u] = gload<uint8_t>(as_global(a.vc.data) + v_at[one] + byte);
                    scale[u] = a.vc.scales[vs_at[one] + g];
                }
#pragma unroll
                for (int u = 0; u < kAttnGenAhead; ++u) {
                    const float4 f = p[min(i + u * strands, (uint32_t)kAttnGenThreads - 1)];
                    const float weight[kAttnGenRows] = {f.x, f.y, f.z, f.w};
                    const float v0 = code_of(w[u], 0) * scale[u], v1 = code_of(w[u], 1) * scale[u];
#pragma unroll
                    for (int r = 0; r < kAttnGenRows; ++r) {
                        o[k][0][r] += mul_or_0(weight[r], v0);
                        o[k][1][r] += mul_or_0(weight[r], v1);
                    }
                }
            }
        }
        __syncthreads();                         // the next tile overwrites p, v_at and red
    }
#pragma unroll
    for (int r = 0; r < kAttnGenRows; ++r) {
        float sum = l[r];
        for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
        if (lane == 0) red[r][wave] = sum;
    }
    // the strands' sums, added in order by the first (q's place is free)
    float* const parts = reinterpret_cast<float*>(q);
    static_assert(sizeof(q) >= kAttnGenThreads * 2 * kAttnGenRows * sizeof(float), "one byte's sums of all threads");
#pragma unroll
    for (int k = 0; k < kAttnGenBytes; ++k) {
        __syncthreads();
        if (strands > 1) {                       // (k is 0 then)
#pragma unroll
            for (int i = 0; i < 2 * kAttnGenRows; ++i) parts[i * kAttnGenThreads + t] = o[k][i & 1][i >> 1];
            __syncthreads();
            if (strand == 0)
#pragma unroll
                for (int i = 0; i < 2 * kAttnGenRows; ++i)
                    for (uint32_t of = 1; of < strands; ++of) o[k][i & 1][i >> 1] += parts[i * kAttnGenThreads + of * cols + t];
        }
        const uint32_t byte = k * kAttnGenThreads + col;
        if (strand != 0 || byte >= v_bytes) continue;
#pragma unroll
        for (int r = 0; r < kAttnGenRows; ++r) {
            if (r >= (int)nr) continue;
            float sum = 0.0f;
            for (int w = 0; w < kAttnGenThreads / 64; ++w) sum += red[r][w];
            const uint32_t s = fast_div(r0 + r, a.rep_div), h = at.head * a.rep + (r0 + r - s * a.rep);
            const uint64_t row = part_row(a, at.part, s, h);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (!a.split)
                    Store<DT>::store1(a.out.data, at.b * a.out.sb + s * a.out.ss + h * a.out.sn + 2 * byte + i, o[k][i][r] * one_over(sum));
                else
                    a.part[row * a.Dv + 2 * byte + i] = o[k][i][r];
            }
            if (a.split && byte == 0) part_stats(a)[row] = make_float2(m[r], sum);
        }
    }
}

// Joins the parts of a row, which are added in a fixed order. Latency is all
// there is to it. Up to 64 parts: a wave a row, a lane a part for the maximum and
// the sum. More: a block takes 32 lanes of a row, half a wave a part, 16 parts at
// a time in as many strands. (32 rows of 256 parts of 128 lanes 7.5 us, one wave
// a row 250; 3200 rows of 16 parts 9.2 by waves.)
constexpr int kJoinThreads = 512;
constexpr int kJoinRows = kJoinThreads / 64;       // of a block, with few parts
constexpr int kJoinLanes = 32;                     // of a block, with many
constexpr int kJoinAhead = 4;                      // parts whose loads go out together
constexpr int kJoinFewParts = 64;                  // of a sequence at most, where waves join rows

template <int DT>
__global__ void __launch_bounds__(kJoinThreads) rope_attn_join_few_kernel(AttnArgs a)
{
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t row = blockIdx.x * kJoinRows + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t b = row / a.part_rows, sh = row - b * a.part_rows;
    const uint32_t s = sh / a.Hq, h = sh - s * a.Hq;
    if (b >= a.B || (int32_t)s >= attn_seq(a, b).count) return;
    const AttnShare share = attn_share<false>(a, b);
    const uint64_t at = (uint64_t)share.first * a.part_rows + sh;
    // a lane a part: the maximum and the sum
    const float2 st = lane < share.n ? part_stats(a)[at + (uint64_t)lane * a.part_rows] : make_float2(kAttnNone, 0.0f);
    float m = st.x;
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    const float weight = part_weight(st.x, m);
    float l = lane < share.n ? st.y * weight : 0.0f;
    for (int d = 1; d < 64; d <<= 1) l += __shfl_xor(l, d);
    const float inv = one_over(l);
    const int64_t out = b * a.out.sb + s * a.out.ss + h * a.out.sn;
    const uint64_t step = (uint64_t)a.part_rows * a.Dv;
    for (uint32_t j = 2 * lane; j < a.Dv; j += 128) {          // (Dv is even)
        const float* part = a.part + at * a.Dv + j;
        float o[2] = {};
        for (uint32_t i = 0; i < share.n; i += kJoinAhead) {
            float2 v[kJoinAhead];
            float w[kJoinAhead];
#pragma unroll
            for (int k = 0; k < kJoinAhead; ++k) {
                const uint32_t one = min(i + k, share.n - 1);
                v[k] = *reinterpret_cast<const float2*>(part + one * step);
                w[k] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, weight), (int)one));
            }
#pragma unroll
            for (int k = 0; k < kJoinAhead; ++k)
                if (i + k < share.n && w[k] != 0.0f) {
                    o[0] = __builtin_fmaf(v[k].x, w[k], o[0]);
                    o[1] = __builtin_fmaf(v[k].y, w[k], o[1]);
                }
        }
        Store<DT>::store1(a.out.data, out + j, o[0] * inv);
        Store<DT>::store1(a.out.data, out + j + 1, o[1] * inv);
    }
}

template <int DT>
__global__ void __launch_bounds__(kJoinThreads) rope_attn_join_many_kernel(AttnArgs a)
{
    constexpr int kStrandsOf = kJoinThreads / kJoinLanes;
    __shared__ float weight[kAttnMaxParts];
    __shared__ float sums[kStrandsOf][kJoinLanes];
    const uint32_t t = threadIdx.x, lane = t & 63;
    const uint32_t b = blockIdx.x / a.part_rows, sh = blockIdx.x - b * a.part_rows, j = blockIdx.y * kJoinLanes + (t & (kJoinLanes - 1)), strand = t / kJoinLanes;
    const uint32_t s = sh / a.Hq, h = sh - s * a.Hq;
    if ((int32_t)s >= attn_seq(a, b).count) return;
    const AttnShare share = attn_share<false>(a, b);
    const uint64_t row = (uint64_t)share.first * a.part_rows + sh;
    const float2* stats = part_stats(a) + row;
    // every wave for itself: the parts' maximum and sum
    float m = kAttnNone, l = 0.0f;
    float2 st[kAttnMaxParts / 64];
#pragma unroll
    for (int k = 0; k < kAttnMaxParts / 64; ++k) {
        const uint32_t i = k * 64 + lane;
        st[k] = i < share.n ? stats[(uint64_t)i * a.part_rows] : make_float2(kAttnNone, 0.0f);
        m = fmaxf(m, st[k].x);
    }
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
#pragma unroll
    for (int k = 0; k < kAttnMaxParts / 64; ++k) {
        const float w = part_weight(st[k].x, m);
        if (k * 64 + lane < share.n) {
            l = __builtin_fmaf(st[k].y, w, l);
            if (t < 64) weight[k * 64 + lane] = w;
        }
    }
    for (int d = 1; d < 64; d <<= 1) l += __shfl_xor(l, d);
    __syncthreads();
    float o = 0.0f;
    const uint64_t step = (uint64_t)a.part_rows * a.Dv;
    const float* part = a.part + row * a.Dv + min(j, a.Dv - 1);
    for (uint32_t i = strand; i < share.n; i += kStrandsOf * kJoinAhead) {
        float v[kJoinAhead];
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k) v[k] = part[min(i + k * kStrandsOf, share.n - 1) * step];
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k) {
            const uint32_t at = i + k * kStrandsOf;
            if (at < share.n && weight[at] != 0.0f) o = __builtin_fmaf(v[k], weight[at], o);
        }
    }
    sums[strand][t & (kJoinLanes - 1)] = o;
    __syncthreads();
    if (t >= kJoinLanes || j >= a.Dv) return;
    o = sums[0][t];
#pragma unroll
    for (int k = 1; k < kStrandsOf; ++k) o += sums[k][t];
    Store<DT>::store1(a.out.data, b * a.out.sb + s * a.out.ss + h * a.out.sn + j, o * one_over(l));
}

}  // namespace
}  // namespace rope
