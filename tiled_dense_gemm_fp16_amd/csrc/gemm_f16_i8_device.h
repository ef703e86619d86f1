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

// What the order says of a workgroup's tile of BM pairs of one expert.
struct I8Tile {
    int expert;      // `experts`: the pairs of none
    int first, rows; // places in `order`
    int tm, tn;
};

__device__ __forceinline__ int i8_start(const I8Args &p, int e) { return min(max(p.starts[e], 0), p.pairs); }

// Find tile `wg` of the grid.  Expert e's pairs make ceil(count / BM) tiles of
// rows; each lane adds up those of neighbouring experts, a scan over the wave
// gives every lane its first one, and the lane whose range holds the tile looks
// for the expert.  (An order whose starts decrease gives tiles that are empty or
// not reached, never places outside of [0, pairs).)  Workgroups past the last
// tile return false.  The remap over XCDs is that of tile_coords, on the tiles
// that there are, so that each XCD has an equal share of them.
template <int BM>
__device__ __forceinline__ bool i8_find_tile(const I8Args &p, int wg, int lane, I8Tile &t)
{
    const int bins = p.experts + 1, per = (bins + 63) / 64;
    const auto tiles_of = [&](int e, int &begin, int &end) {
        begin = i8_start(p, e);
        end = e < p.experts ? i8_start(p, e + 1) : p.pairs;
        return max(0, end - begin + BM - 1) / BM;
    };
    int begin, end, mine = 0;
    for (int i = 0; i < per; ++i)
        if (lane * per + i < bins)
            mine += tiles_of(lane * per + i, begin, end);
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int other = __shfl_up(upto, d);
        upto += lane >= d ? other : 0;
    }
    const int tiles_m = min(__builtin_amdgcn_readlane(upto, 63), p.tiles_m), total = tiles_m * p.tiles_n;
    // (an XCD's share, and this workgroup's place in it)
    const int share = total / 8 + (wg % 8 < total % 8 ? 1 : 0);
    if (wg / 8 >= share)
        return false;
    const int id = wg % 8 * (total / 8) + min(wg % 8, total % 8) + wg / 8;
    constexpr int kGroup = 4;
    const int width = kGroup * p.tiles_n, group = id / width, in_group = id - group * width;
    const int high = min(tiles_m - group * kGroup, kGroup);
    t.tm = group * kGroup + in_group % high;
    t.tn = in_group / high;
    const int owner = __ffsll((unsigned long long)__ballot(upto > t.tm)) - 1;   // the first whose range ends behind the tile
    int expert = 0, first = 0, rows = 0, at = upto - mine;
    if (lane == owner)
        for (int i = 0; i < per && lane * per + i < bins; ++i) {
            const int n = tiles_of(lane * per + i, begin, end);
            if (t.tm < at + n) {
                expert = lane * per + i;
                first = begin + (t.tm - at) * BM;
                rows = min(BM, end - first);
                break;
            }
            at += n;
        }
    t.expert = __builtin_amdgcn_readlane(expert, owner);
    t.first = __builtin_amdgcn_readlane(first, owner);
    t.rows = __builtin_amdgcn_readlane(rows, owner);
    return true;
}

// The pair at place `i` of a tile's rows, -1 past them or where order does not
// name one.
__device__ __forceinline__ int i8_pair(const I8Args &p, const I8Tile &t, int i)
{
    if (i >= t.rows)
        return -1;
    const int pair = p.order[t.first + i];
    return pair >= 0 && pair < p.pairs ? pair : -1;
}

} // namespace gemm_f16_impl

#endif
