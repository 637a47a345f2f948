// rope_proj_lora_fwd: a head projection shared by many requests, each token
// with its own low-rank adapter, and a rotary epilogue.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <string>

#include "rope_host.hpp"
#include "rope_lora_kernels.hpp"
#include "rope_plan.hpp"
#include "rope_proj_host.hpp"

namespace rope {
namespace {

// Whether the few-token kernel (blocks of 64 tokens by 32 output lanes) is
// taken for more tokens than kLoraFewTokens too: it has no sort and fills the
// chip sooner, but its adapters' part, and h before it, are dot products that
// grow with the rank R: it takes as long as blocks * (1 + R/192) + M * R/256
// blocks without adapters would, and tiles as long as 960 of them. Measured on
// MI355X (8 adapters, each token its own, weights from memory; us here and on
// tiles, both with the launches before them):
//   blocks:     R 8                     R 32                    R 128
//   K 1536, 192 lanes:
//     120       22, 61                  33, 64                  77, 81
//     240       26, 61                  44, 65                  118, 90
//     564       57, 66                  101, 70                 264, 105
//   K 1536, 2048 lanes:
//     320       31, 63                  40, 68                  75, 87
//     640       42, 65                  57, 69                  113, 89
//     1280      68, 64                  92, 67                  182, 88
//   K 1536, 5120 lanes:
//     480       31, 63                  39, 68                  71, 91
//     800       55, 64                  71, 69                  128, 88
// Without adapters 640 blocks of these take 34 and 45, 800 47 and 44, 1280 57
// and 47. K of 512 and 4096 meet within a fifth of the same sums (2048 lanes, R
// 128: 320 blocks 55 and 58, 121 and 155; 640 blocks 80 and 60, 186 and 158).
// One adapter for all tokens is up to a quarter quicker here, 100 adapters up
// to a third slower. Of 266 calls measured the rule picks the slower kernel for
// 10, at worst 1.24 times the other's time. (Up to 64 tokens the tiles are
// mostly empty: K 1536, 24576 lanes, 64 tokens, R 8 of 64 adapters 47 and 138,
// one adapter of R 128 65 and 62, 64 of these 275 and 245; every narrower call
// is quicker here.)
bool few_for_more(int64_t blocks, int64_t M, int64_t R)
{
    return blocks * (768 + 4 * R) + 3 * M * R <= 960 * 768;
}

// A grid's second dimension counts the few-token kernel's 64-token blocks;
// calls of more tokens that no tiled kernel takes go to the general one.
constexpr int64_t kFewTokensMax = 64 * 65535ll;

// A call's checked plan and what is launched for it.
struct LoraLaunch {
    ProjLaunch P;
    LoraArgs l{};
    int heads = 0;
    bool tiles = false;      // the tiled projection kernels
    bool few = false;        // else the kernel for few tokens, else the general one
    FewArgs units{};         // its fragments
};

rope_status_t prepare_lora(void* y, rope_dtype_t y_dtype, const void* x, const void* w, rope_dtype_t dtype,
                           const int64_t y_shape[4], int64_t K, const rope_lora_t* lora,
                           const void* r1, const int64_t r1_shape[4], const int64_t r1_strides[4],
                           const void* r2, const int64_t r2_shape[4], const int64_t r2_strides[4],
                           rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2], void* workspace,
                           int64_t workspace_bytes, LoraLaunch* L, std::string* why)
{
    const LoraCheck c{lora, workspace, workspace_bytes};
    ProjPlan& q = L->P.q;
    rope_status_t st = make_proj_plan(y, y_dtype, x, w, dtype, y_shape, K, r1, r1_shape, r1_strides, r2, r2_shape,
                                      r2_strides, table_dtype, mode, partial_slice, &q, why, &c);
    if (st != ROPE_OK || q.noop) return st;
    if ((st = plan_proj_kernel(&L->P, why)) != ROPE_OK) return st;
    const Plan& p = q.rope;
    L->heads = (int)p.N;
    LoraArgs& l = L->l;
    if (lora->count > 0 && lora->rank > 0) {
        l.a = static_cast<const uint16_t*>(lora->a);
        l.b = static_cast<const uint16_t*>(lora->b);
        l.ids = lora->adapters;
        l.scales = lora->scales;
        l.h = static_cast<float*>(workspace);
        l.count = (int32_t)lora->count;
        l.R = (int32_t)lora->rank;
    }
    // the kernel for few tokens: adjacent pairs that start on an even lane,
    // or partners whole fragments apart
    const ProjArgs& a = L->P.a;
    FewArgs& u = L->units;
    u.head_units = a.Dh / 32;
    u.apart = a.L > 0 && a.half > 1;
    if (u.apart) {
        u.first_frag = a.start / 16;
        u.slice_frags = a.L / 16;
        u.half_frags = a.half / 16;
        u.slice_units = u.slice_frags / 2;
    }
    const bool units = u.apart ? a.start % 16 == 0 && a.half % 16 == 0 : a.start % 2 == 0;
    // the tiled kernels need each rotation group within one tile, and, with
    // adapters, sorted rows: their tiles for a bound on these
    const bool fits = L->P.sq || proj_groups_in_tiles(p.D, p.start, p.L, a.half);
    const int64_t few_blocks = (a.M + 63) / 64 * (a.N / 32);
    L->tiles = fits && a.M > kLoraFewTokens && l.count <= kLoraSortAdapters &&
               !(units && few_for_more(few_blocks, a.M, l.R));
    if (L->tiles && l.count > 0) {
        const int64_t MB = (lora_row_bound(a.M, l.count) + L->P.BM - 1) / L->P.BM;
        if (MB * a.NB > (int64_t)(kMaxGridItems / (uint64_t)L->P.threads)) L->tiles = false;
        else L->P.grid = (uint32_t)(MB * a.NB);
    }
    L->few = !L->tiles && units && a.M <= kFewTokensMax;
    return ROPE_OK;
}

// The tiled kernels, with adapters (ARGS LoraProjArgs) or without.
template <int DT, int TT, class ARGS>
void launch_tiles(const ProjLaunch& P, const ARGS& a, hipStream_t s)
{
    const dim3 grid(P.grid), block((uint32_t)P.threads);
    if (P.sq) {
        switch (a.epi) {
        case 0: hipLaunchKernelGGL((rope_proj_sq_kernel<DT, TT, 0, ARGS>), grid, block, 0, s, a); break;
        case 1: hipLaunchKernelGGL((rope_proj_sq_kernel<DT, TT, 1, ARGS>), grid, block, 0, s, a); break;
        default: hipLaunchKernelGGL((rope_proj_sq_kernel<DT, TT, -1, ARGS>), grid, block, 0, s, a); break;
        }
    } else if (P.BN == 192) {
        hipLaunchKernelGGL((rope_proj_kernel<DT, 192, TT, ARGS>), grid, block, 0, s, a);
    } else {
        hipLaunchKernelGGL((rope_proj_kernel<DT, 128, TT, ARGS>), grid, block, 0, s, a);
    }
}

template <int DT, class ARGS>
void launch_tiles_tt(const ProjLaunch& P, const ARGS& a, hipStream_t s)
{
    switch (P.tdt) {
    case ROPE_DTYPE_F32: return launch_tiles<DT, ROPE_DTYPE_F32>(P, a, s);
    case ROPE_DTYPE_F16: return launch_tiles<DT, ROPE_DTYPE_F16>(P, a, s);
    default: return launch_tiles<DT, ROPE_DTYPE_BF16>(P, a, s);
    }
}

// Tokens of a block of the few-token kernel, in 16s.
int few_tiles(int32_t M) { return M <= 16 ? 1 : M <= 32 ? 2 : 4; }

// Blocks of the general kernel.
uint32_t head_blocks(const LoraLaunch& L)
{
    const uint64_t tiles = (uint64_t)((L.P.a.M + kHeadTokens - 1) / kHeadTokens) * (uint64_t)L.heads;
    return (uint32_t)std::min<uint64_t>(tiles, kMaxGridItems / 256);
}

template <int DT, int MT>
void launch_few(const FewArgs& a, int tdt, hipStream_t s)
{
    const dim3 grid((uint32_t)(a.N / 32), (uint32_t)((a.M + 16 * MT - 1) / (16 * MT)));
    hipLaunchKernelGGL((rope_lora_few_kernel<DT, MT>), grid, dim3(64 * kFewWaves), 0, s, a, tdt);
}

template <int DT>
hipError_t launch_lora(const LoraLaunch& L, hipStream_t s)
{
    LoraProjArgs a;
    static_cast<ProjArgs&>(a) = L.P.a;
    a.l = L.l;
    if (a.l.count > 0) {
        if (L.tiles) {
            // rows in the order of their adapters, in the workspace behind h
            const int64_t bound = lora_row_bound(a.M, a.l.count), places = bound + kLoraTileRows;
            int32_t* order = reinterpret_cast<int32_t*>(a.l.h + (int64_t)a.M * a.l.R);
            int32_t* group_ids = order + places;
            int32_t* rows = group_ids + places / 32 + 1;
            hipLaunchKernelGGL(rope_lora_sort_kernel, dim3(1), dim3(kSortThreads), 0, s, a.l.ids, a.l.count, a.M, order,
                               group_ids, rows);
            hipError_t err = hipGetLastError();
            if (err != hipSuccess) return err;
            a.l.order = order;
            a.l.group_ids = group_ids;
            a.l.rows = rows;
            // (x has fewer than 2^31 elements: 2^25 tokens at most, 2^20 groups)
            hipLaunchKernelGGL((rope_lora_shrink_tile_kernel<DT>),
                               dim3((uint32_t)((bound + 31) / 32), (uint32_t)(a.l.R + 31) / 32),
                               dim3(64 * kShrinkTileWaves), 0, s, a.l, a.x, a.K);
            err = hipGetLastError();
            if (err != hipSuccess) return err;
        } else {
            hipLaunchKernelGGL((rope_lora_shrink_kernel<DT>),
                               dim3((uint32_t)std::min<uint64_t>((uint64_t)a.M, kMaxGridItems / (64 * kShrinkWaves)),
                                    (uint32_t)(a.l.R + kShrinkWaves - 1) / kShrinkWaves),
                               dim3(64 * kShrinkWaves), 0, s, a.l, a.x, a.M, a.K);
            const hipError_t err = hipGetLastError();
            if (err != hipSuccess) return err;
        }
    }
    if (L.tiles && a.l.count > 0) {
        launch_tiles_tt<DT>(L.P, a, s);
    } else if (L.tiles) {
        launch_tiles_tt<DT>(L.P, static_cast<const ProjArgs&>(a), s);
    } else if (L.few) {
        FewArgs f = L.units;
        static_cast<LoraProjArgs&>(f) = a;
        switch (few_tiles(a.M)) {
        case 1: launch_few<DT, 1>(f, L.P.tdt, s); break;
        case 2: launch_few<DT, 2>(f, L.P.tdt, s); break;
        default: launch_few<DT, 4>(f, L.P.tdt, s); break;
        }
    } else {
        hipLaunchKernelGGL((rope_lora_head_kernel<DT>), dim3(head_blocks(L)), dim3(256), 0, s, a, L.P.tdt, L.heads);
    }
    return hipGetLastError();
}

}  // namespace
}  // namespace rope

extern "C" {

rope_status_t rope_proj_lora_fwd(
    void* y, rope_dtype_t y_dtype, const void* x, const void* w, rope_dtype_t dtype,
    const int64_t y_shape[4], int64_t K, const rope_lora_t* lora,
    const void* r1, const int64_t r1_shape[4], const int64_t r1_strides[4],
    const void* r2, const int64_t r2_shape[4], const int64_t r2_strides[4],
    rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* workspace, int64_t workspace_bytes, void* stream)
{
    rope::LoraLaunch L;
    std::string why;
    rope_status_t st = rope::prepare_lora(y, y_dtype, x, w, dtype, y_shape, K, lora, r1, r1_shape, r1_strides, r2,
                                          r2_shape, r2_strides, table_dtype, mode, partial_slice, workspace,
                                          workspace_bytes, &L, &why);
    if (st != ROPE_OK) return rope::set_error(st, why);
    if (L.P.q.noop) return ROPE_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t err = L.P.q.in_dtype == ROPE_DTYPE_BF16 ? rope::launch_lora<ROPE_DTYPE_BF16>(L, s)
                                                           : rope::launch_lora<ROPE_DTYPE_F16>(L, s);
    if (err != hipSuccess)
        return rope::set_error(ROPE_ERR_RUNTIME, std::string("kernel launch: ") + hipGetErrorString(err));
    return ROPE_OK;
}

rope_status_t rope_proj_lora_launch_info(rope_dtype_t y_dtype, rope_dtype_t dtype, const int64_t y_shape[4], int64_t K,
                                         int64_t count, int64_t rank, const void* r1, const int64_t r1_shape[4],
                                         const int64_t r1_strides[4], const void* r2, const int64_t r2_shape[4],
                                         const int64_t r2_strides[4], rope_dtype_t table_dtype, int64_t mode,
                                         const int64_t partial_slice[2], int64_t info[ROPE_LAUNCH_INFO_LEN])
{
    if (info == nullptr) return rope::set_error(ROPE_ERR_NULLPTR, "info is NULL");
    for (int i = 0; i < ROPE_LAUNCH_INFO_LEN; ++i) info[i] = 0;
    // distinct, 16-byte aligned stand-ins, never dereferenced
    const auto nowhere = [](int i) { return reinterpret_cast<void*>(uint64_t(i) << 60); };
    const rope_lora_t lora{nowhere(5), nowhere(8), static_cast<const int32_t*>(nowhere(11)), nullptr, count, rank};
    rope::LoraLaunch L;
    std::string why;
    rope_status_t st = rope::prepare_lora(nowhere(2), y_dtype, nowhere(3), nowhere(4), dtype, y_shape, K, &lora, r1,
                                          r1_shape, r1_strides, r2, r2_shape, r2_strides, table_dtype, mode,
                                          partial_slice, nowhere(12), int64_t(1) << 60, &L, &why);
    if (st != ROPE_OK) return rope::set_error(st, why);
    const rope::ProjLaunch& P = L.P;
    if (P.q.noop) return ROPE_OK;
    if (L.tiles) {
        info[0] = P.sq ? ROPE_KERNEL_PROJ_SQUARE : ROPE_KERNEL_PROJ_HEADS;
        info[1] = P.grid;
        info[2] = P.threads;
        info[3] = P.BM;
        info[4] = P.BN;
        info[5] = P.sq && P.a.epi >= 0 ? 1 + P.a.epi : 0;
        info[6] = P.sq && P.a.epi >= 0 && P.q.rope.L > 0 && P.a.tab_crl >= 0 ? 1 : 0;
        info[7] = L.l.count > 0 ? 1 : 0;
    } else if (L.few) {
        const int64_t tokens = 16 * rope::few_tiles(P.a.M);
        info[0] = ROPE_KERNEL_PROJ_FEW;
        info[1] = P.a.N / 32 * ((P.a.M + tokens - 1) / tokens);
        info[2] = 64 * rope::kFewWaves;
        info[3] = tokens;
        info[4] = 32;
    } else {
        info[0] = ROPE_KERNEL_PROJ_GENERAL;
        info[1] = rope::head_blocks(L);
        info[2] = 256;
        info[3] = rope::kHeadTokens;
        info[4] = P.a.Dh;
    }
    return ROPE_OK;
}

int64_t rope_proj_lora_workspace(const int64_t y_shape[4], int64_t K, int64_t rank)
{
    if (y_shape == nullptr || K <= 0 || rank <= 0 || rank > ROPE_LORA_RANK_MAX || y_shape[0] <= 0 || y_shape[1] <= 0)
        return 0;
    int64_t M;
    if (__builtin_mul_overflow(y_shape[0], y_shape[1], &M)) return 0;
    const int64_t n = rope::lora_workspace_bytes(M, rank);
    return n < 0 ? 0 : n;
}

}  // extern "C"
