// gemm_f16_i8_internal.h -- shared between the host API of the 8-bit operators
// and the routed experts (gemm_f16_i8_api.cpp) and their kernels.  Not part of
// the public ABI.
#ifndef GEMM_F16_I8_INTERNAL_H
#define GEMM_F16_I8_INTERNAL_H

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_f16_i8.h"
#include "gemm_f16_internal.h"

namespace gemm_f16_impl {

// A compiled configuration of the product.
struct I8Config {
    const char *name;
    int block_m, block_n;
    int waves;
    int stages;   // LDS stages of 128 bytes of k; 0: the kernel for few rows, which takes its operands straight from memory
    int resident; // workgroups of a CU, by LDS and registers
    // us of a step of k (the kernel for few rows: of 8 steps, one for each of its
    // waves) and of the rest of a tile, dense and over experts (see estimate())
    float step, fixed, experts_step, experts_fixed;
};
constexpr int kI8BlockK = 128;       // k of a tile's step
constexpr int kI8StreamK = 256;      // k of a step of the kernel for few rows
constexpr int kNumI8Configs = 11;
extern const I8Config kI8Configs[kNumI8Configs];

// LDS of a workgroup that works in tiles: the stages, a factor for each row and a scale
// for each column, and over experts each row's pair.  (A tile of C on its way out
// fits into the stages, and the quarters of a tile take less than all of it.)
constexpr int i8_lds_bytes(int block_m, int block_n, int stages, bool experts)
{
    return stages * (block_m + block_n) * kI8BlockK + 4 * ((experts ? 2 : 1) * block_m + block_n);
}

// The largest tile: where its last round over the 256 CUs has kI8Cut tiles or
// fewer, those are cut into quarters of 128 x 128.  How many are not:
constexpr int kI8Cut = 128;
__host__ __device__ inline int i8_uncut(int tiles) { return tiles % 256 <= kI8Cut ? tiles - tiles % 256 : tiles; }

struct I8Args {
    const int8_t *A, *W;
    const float *a_scales, *w_scales;
    _Float16 *C;
    int *partial;          // a split's sums: splits x M x N; null unless split
    int64_t a_pitch, w_pitch;   // bytes, at most 2^22
    int M, N, K;           // M rows of A; K rounded up to a multiple of 16
    int tiles_m, tiles_n;  // (experts: tiles_m is what the grid has room for)
    int splits, k_split;   // k of a split, a multiple of the configuration's step; >= K unless split
    int uncut;             // the largest tile: its workgroups for whole tiles, those behind are for quarters of tiles
    float alpha;
    int relu;
    int vec_c;             // 8: C's rows take 16-byte stores; 4: 8-byte; 1: 2-byte
    // experts: W is experts x N rows, and C has a row for each pair
    const int32_t *order, *starts;
    int experts, pairs, pairs_per_row;
};

hipError_t launch_i8(int config, const I8Args &a, int64_t grid, hipStream_t s);
hipError_t launch_i8_experts(int config, const I8Args &a, int64_t grid, hipStream_t s);
// C = rne16(epi(alpha a_scales w_scales (sum of the splits' partial sums)))
hipError_t launch_i8_reduce(const I8Args &a, hipStream_t s);

hipError_t launch_i8_compress(const _Float16 *X, int64_t stride, int8_t *codes, int64_t pitch, float *scales, int64_t rows,
                              int64_t K, hipStream_t s);
hipError_t launch_i8_expand(const int8_t *codes, int64_t pitch, const float *scales, _Float16 *X, int64_t rows, int64_t K,
                            hipStream_t s);

struct RouteArgs {
    const void *logits;
    const float *bias;
    int32_t *ids;
    float *weights;
    int64_t stride;
    int tokens, experts, top_k, half, sigmoid, groups, top_groups, renormalise;
    float scale;
    // made by launch_route(): experts of a group, 2^22 over that, and log2 of the lanes of a group
    int group_size, team_shift;
    unsigned group_magic;
};
hipError_t launch_route(const RouteArgs &a, hipStream_t s);
hipError_t launch_expert_order(const int32_t *ids, int32_t *order, int32_t *starts, int pairs, int experts, hipStream_t s);
hipError_t launch_expert_sum(const _Float16 *Y, const float *weights, _Float16 *out, int64_t tokens, int top_k, int64_t N,
                             hipStream_t s);

} // namespace gemm_f16_impl

#endif
