// gemm_f16_i8_device.h -- device code that the kernels of the 8-bit products
// share: which rows a workgroup has, and the last steps of a sum.
#ifndef GEMM_F16_I8_DEVICE_H
#define GEMM_F16_I8_DEVICE_H

#include "gemm_f16_i8_internal.h"
#include "gemm_f16_tile.h"

namespace gemm_f16_impl {

__device__ __forceinline__ int4v i8_mfma(int4v x, int4v y, int4v acc)
{
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(x, y, acc, 0, 0, 0);
}

// The fp32 factor of a row is (alpha a_scale); a sum times it and a column's
// scale, through the epilogue.  (Adding 0 makes +0 of the -0 that a sum of 0 has
// under a negative factor.)
__device__ __forceinline__ half_t i8_out(int sum, float row, float column, int relu)
{
    float v = __builtin_fmaf((float)sum, row * column, 0.0f);
    if (relu)
        v = __builtin_fmaxf(v, 0.0f);
    return (half_t)v;
}

// A workgroup's tile: rows of A from `first` on (experts: of those that the
// places from `first` on in `order` name), columns from n0 on.
struct I8Tile {
    int first, rows, n0;
    int expert;      // `experts`: the pairs of none
};

// Tile `id` of a product: four rows of tiles at a time, so that tiles which run
// together share panels of both operands.
__device__ __forceinline__ void i8_walk(int id, int tiles_m, int tiles_n, int &tm, int &tn)
{
    constexpr int kGroup = 4;
    const int width = kGroup * tiles_n, group = id / width, in_group = id - group * width;
    const int high = min(tiles_m - group * kGroup, kGroup);
    tm = group * kGroup + in_group % high;
    tn = in_group / high;
}

// The place in 0 .. count - 1 of workgroup `wg`, an equal share of neighbouring
// ones for each XCD (workgroups are handed to them in turn); count for none.
__device__ __forceinline__ int i8_place(int wg, int count)
{
    const int xcd = wg % 8, share = count / 8 + (xcd < count % 8 ? 1 : 0);
    return wg / 8 < share ? xcd * (count / 8) + min(xcd, count % 8) + wg / 8 : count;
}

// Inclusive sums over the wave, in the vector unit's own lane moves.
__device__ __forceinline__ int wave_prefix(int x)
{
#define GEMM_F16_STEP(CTRL, ROWS) x += __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, false)
    GEMM_F16_STEP(0x111, 0xf);   // row_shr:1, 2, 4, 8
    GEMM_F16_STEP(0x112, 0xf);
    GEMM_F16_STEP(0x114, 0xf);
    GEMM_F16_STEP(0x118, 0xf);
    GEMM_F16_STEP(0x142, 0xa);   // row_bcast:15, :31
    GEMM_F16_STEP(0x143, 0xc);
#undef GEMM_F16_STEP
    return x;
}

// Find the tile of workgroup `wg`.  Expert e's pairs make ceil(count / BM) tiles of
// rows; each lane adds up those of EACH neighbouring experts, a scan over the
// wave gives every lane its first one, and the lane whose range holds the tile
// looks for the expert.  (An order whose starts decrease gives tiles that are
// empty or not reached, never places outside of [0, pairs).)  Workgroups without a
// tile return false.  CUT: the tiles of a last round may be cut in quarters, for
// the workgroups from p.uncut on; `quarter` is set for them.
template <int BM, int BN, bool CUT, int EACH>
__device__ __forceinline__ bool i8_search(const I8Args &p, int wg, int lane, I8Tile &t, bool &quarter)
{
    int start[EACH + 1], n[EACH], mine = 0;   // experts EACH lane, ...: their starts and numbers of tiles
    // (buffer loads and no choice between values: all are in flight together)
    const __amdgpu_buffer_rsrc_t starts = make_rsrc(p.starts, (uint32_t)(p.experts + 1) * 4u);
#pragma unroll
    for (int i = 0; i <= EACH; ++i)
        start[i] = __builtin_amdgcn_raw_buffer_load_b32(starts, (uint32_t)(lane * EACH + i) * 4u, 0, 0);
#pragma unroll
    for (int i = 0; i <= EACH; ++i)
        start[i] = max(min(max(start[i], 0), p.pairs), lane * EACH + i > p.experts ? p.pairs : 0);
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        n[i] = (max(0, start[i + 1] - start[i]) + BM - 1) / BM;
        mine += n[i];
    }
    const int upto = wave_prefix(mine);
    const int tiles_m = min(__builtin_amdgcn_readlane(upto, 63), p.tiles_m), total = tiles_m * p.tiles_n;
    int id, part = 0;
    quarter = CUT && wg >= p.uncut;
    if (quarter) {   // the quarters of a tile to one XCD
        const int w = wg - p.uncut;
        id = i8_uncut(total) + w % 8 + w / 32 * 8;
        part = w / 8 % 4;
        if (id >= total)
            return false;
    } else {
        const int count = CUT ? i8_uncut(total) : total;
        id = i8_place(wg, count);
        if (id >= count)
            return false;
    }
    int tm, tn;
    i8_walk(id, tiles_m, p.tiles_n, tm, tn);
    const int owner = __ffsll((unsigned long long)__ballot(upto > tm)) - 1;   // the first whose range ends behind the tile
    int expert = 0, first = 0, rows = 0, at = upto - mine;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        if (tm >= at && tm < at + n[i]) {
            expert = lane * EACH + i;
            first = start[i] + (tm - at) * BM;
            rows = min(BM, start[i + 1] - first);
        }
        at += n[i];
    }
    t.expert = __builtin_amdgcn_readlane(expert, owner);
    t.first = __builtin_amdgcn_readlane(first, owner);
    t.rows = __builtin_amdgcn_readlane(rows, owner);
    t.n0 = tn * BN;
    if (quarter) {
        t.first += part / 2 * (BM / 2);
        t.rows = min(t.rows - part / 2 * (BM / 2), BM / 2);
        t.n0 += part % 2 * (BN / 2);
        return t.rows > 0 && t.n0 < p.N;
    }
    return true;
}

// (65 places for 64 lanes: the pairs of none come behind the last expert)
template <int BM, int BN, bool CUT>
__device__ __forceinline__ bool i8_find_tile(const I8Args &p, int wg, int lane, I8Tile &t, bool &quarter)
{
    return p.experts < 128   ? i8_search<BM, BN, CUT, 2>(p, wg, lane, t, quarter)
           : p.experts < 320 ? i8_search<BM, BN, CUT, 5>(p, wg, lane, t, quarter)
                             : i8_search<BM, BN, CUT, 17>(p, wg, lane, t, quarter);
}

// The pair at place `i` of a tile's rows, -1 past them or where order does not
// name one.
__device__ __forceinline__ int i8_pair(const I8Args &p, const I8Tile &t, int i)
{
    const int pair = p.order[min(t.first + i, p.pairs - 1)];
    return i < t.rows && pair >= 0 && pair < p.pairs ? pair : -1;
}

} // namespace gemm_f16_impl

#endif
