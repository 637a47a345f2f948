// rope_proj_host.hpp -- the launch plan of a projection: its kernel
// arguments, tile and epilogue. Included next to the host code that launches
// the kernels of rope_proj_kernels.hpp.
#pragma once

#include <string>

#include "rope_host.hpp"
#include "rope_proj_kernels.hpp"

namespace rope {
namespace {

// A projection call's checked plan, kernel arguments and kernel choice.
struct ProjLaunch {
    ProjPlan q;
    ProjArgs a{};
    bool sq = false;            // square 256 x 256 tiles (else tiles of whole heads)
    int BM = 0, BN = 0, threads = 0;
    uint32_t grid = 0;
    int tdt = ROPE_DTYPE_BF16;  // table type the kernel is instantiated for
};

// Fill the kernel arguments and choose the kernel of the checked plan P->q.
rope_status_t plan_proj_kernel(ProjLaunch* P, std::string* why)
{
    const ProjPlan& q = P->q;
    const Plan& p = q.rope;
    ProjArgs& a = P->a;
    a.x = static_cast<const uint16_t*>(q.x);
    a.w = static_cast<const uint16_t*>(q.w);
    a.y = q.y;
    a.ydt = q.out_dtype;
    a.r1 = p.r1;
    a.r2 = p.r2;
    a.t1b = p.t1[0]; a.t1s = p.t1[1]; a.t1n = p.t1[2];
    a.t2b = p.t2[0]; a.t2s = p.t2[1]; a.t2n = p.t2[2];
    // the plan bounds x and w below 2^31 elements, so M, N and K fit in 32 bits
    a.M = (int32_t)(p.B * p.S);
    a.N = (int32_t)(p.N * p.D);
    a.K = (int32_t)q.K;
    a.S = (int32_t)p.S;
    a.Dh = (int32_t)p.D;
    a.start = (int32_t)p.start;
    a.L = (int32_t)p.L;
    a.half = p.L > 0 ? (int32_t)p.half : 1;
    // Square 256 x 256 tiles when K is a whole number of stage pairs (128 k)
    // and every rotation group lies within one 256-lane column tile;
    // otherwise tiles of whole heads, or of part of one wider head: 192 lanes
    // (384 tokens) for heads of a multiple of 3 lanes, else 128 lanes (256
    // tokens).
    const bool sq = P->sq = a.K % (2 * kProjBK) == 0 &&
                    proj_groups_in_column_tiles(p.D, (int64_t)a.N, p.start, p.L, a.half, ProjSq::BN);
    const int BN = P->BN = sq ? ProjSq::BN : (int)proj_tile_lanes(p.D);
    const int BM = P->BM = sq ? ProjSq::BM : BN == 192 ? ProjTile<192>::BM : ProjTile<128>::BM;
    const int threads = P->threads = sq ? ProjSq::THREADS : BN == 192 ? ProjTile<192>::THREADS : ProjTile<128>::THREADS;
    const int64_t MB = (a.M + BM - 1) / BM, NB = (a.N + BN - 1) / BN;
    // the dispatch packet holds the grid in work-items as a 32-bit number
    if (MB * NB > (int64_t)(0xFFFFFFFFull / threads))
    {
        *why = "the projection's grid exceeds one launch";
        return ROPE_ERR_UNSUPPORTED;
    }
    a.MB = (int32_t)MB;
    a.NB = (int32_t)NB;
    // Measured on MI355X on the (4*4096 tokens, 1536) x (24576, 1536) MLA
    // projection: groups of 4 M-tiles with each XCD taking a contiguous run
    // of tiles.
    a.group_m = 4;
    a.xcd_chunk = (int32_t)(MB * NB / 8);
    a.s_div = make_fastdiv((uint32_t)p.S);
    a.dh_div = make_fastdiv((uint32_t)p.D);
    // The vector epilogue: whole 8-lane slice vectors whose partners are in
    // the vector or a whole vector away, and 16-byte aligned runs of 8 cos
    // and 8 sin values in every table row.
    {
        const int64_t per = 16 / p.tesize;                 // table lanes per 16 bytes
        bool f = p.L > 0 && p.start % 8 == 0 && p.L % 8 == 0 && (p.half == 1 || p.half % 8 == 0);
        f = f && aligned16(p.r1) && aligned16(p.r2);
        for (int k = 0; k < 3 && f; ++k) f = p.t1[k] % per == 0 && p.t2[k] % per == 0;
        a.fast = f ? 1 : 0;
    }
    // The square tiles' epilogue: the vector epilogue when the slice is
    // whole vectors (fast) whose partners are in the vector (interleave) or
    // whole vectors away within one wave's 128 lanes, with the tables' rows
    // staged in LDS when both tables are shared by all heads and a row's L
    // values take 16, 32, 64 or 128 bytes that 32-bit byte offsets reach;
    // otherwise the general one.
    a.epi = -1;
    a.tab_crl = -1;
    if (sq) {
        if (p.L == 0) {
            a.epi = 0;
        } else if (a.fast && (a.half == 1 || proj_groups_in_column_tiles(p.D, (int64_t)a.N, p.start, p.L, a.half,
                                                                          ProjSq::BN / 2))) {
            a.epi = a.half == 1 ? 0 : 1;
            if (p.t1[2] == 0 && p.t2[2] == 0) {
                const int64_t row = p.L * p.tesize;
                int crl = -1;
                for (int k = 0; k < 4; ++k)
                    if (row == (int64_t)16 << k) crl = k;
                const int64_t reach1 = ((p.B - 1) * p.t1[0] + (p.S - 1) * p.t1[1] + p.L) * p.tesize;
                const int64_t reach2 = ((p.B - 1) * p.t2[0] + (p.S - 1) * p.t2[1] + p.L) * p.tesize;
                if (crl >= 0 && reach1 <= (int64_t)UINT32_MAX && reach2 <= (int64_t)UINT32_MAX) a.tab_crl = crl;
            }
        }
    }
    P->grid = (uint32_t)(MB * NB);
    P->tdt = p.L > 0 ? p.tdtype : (int)ROPE_DTYPE_BF16;
    return ROPE_OK;
}

}  // namespace
}  // namespace rope
