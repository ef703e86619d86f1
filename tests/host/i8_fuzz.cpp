// i8_fuzz.cpp -- host-only driver for the validation and planning of the 8-bit
// and expert entry points, built with AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_host_i8_sanitized.py.  The kernel
// launchers are replaced by stubs that check what reaches them: sizes, offsets
// and grids within what the kernels assume, splits that cover K without an
// empty one.  Pointers are stand-ins that nothing dereferences.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "gemm_f16_i8_internal.h"

static int g_launches = 0, g_fails = 0;
#define CHECK(cond)                                                       \
    do {                                                                  \
        if (!(cond)) {                                                    \
            ++g_fails;                                                    \
            if (g_fails < 20)                                             \
                printf("failed: %s (line %d)\n", #cond, __LINE__);        \
        }                                                                 \
    } while (0)

namespace gemm_f16_impl {
bool overlaps(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes)
{
    if (a_bytes <= 0 || b_bytes <= 0)
        return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + (uintptr_t)b_bytes && b0 < a0 + (uintptr_t)a_bytes;
}
gemm_f16_status_t check_device(int *device)
{
    *device = 0;
    return GEMM_F16_SUCCESS;
}
static void check_args(int config, const I8Args &a, int64_t grid)
{
    ++g_launches;
    const I8Config &d = kI8Configs[config];
    CHECK(config >= 0 && config < kNumI8Configs && grid > 0 && grid * 64 * d.waves <= 0xffffffff);
    CHECK(a.N > 0 && a.K >= 0 && a.K % 16 == 0 && a.K <= 1 << 17 && a.C && a.a_scales && a.w_scales && (a.K == 0 || (a.A && a.W)));
    CHECK(a.a_pitch >= a.K && a.w_pitch >= a.K && a.a_pitch % 16 == 0 && a.w_pitch % 16 == 0 && a.a_pitch <= 1 << 22 && a.w_pitch <= 1 << 22);
    CHECK((int64_t)d.block_n * a.w_pitch < (int64_t)1 << 31);
    CHECK(a.vec_c == 1 || (a.N % a.vec_c == 0 && (uintptr_t)a.C % (2 * a.vec_c) == 0));
    CHECK((int64_t)a.tiles_n * d.block_n >= a.N && (int64_t)(a.tiles_n - 1) * d.block_n < a.N);
}
hipError_t launch_i8(int config, const I8Args &a, int64_t grid, hipStream_t)
{
    check_args(config, a, grid);
    const I8Config &d = kI8Configs[config];
    const int step = d.stages > 0 ? kI8BlockK : kI8StreamK;
    const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
    CHECK(a.M > 0 && (int64_t)a.tiles_m * d.block_m >= a.M);
    if (d.block_m == 256 && d.block_n == 256 && a.splits == 1) {   // a last round in quarters, for all of its tiles
        CHECK(a.uncut <= tiles && tiles - a.uncut <= kI8Cut && (a.uncut == tiles || a.uncut % 256 == 0));
        CHECK(a.uncut == tiles ? grid == tiles : grid - a.uncut == 4 * 8 * ((tiles - a.uncut + 7) / 8));
    } else {
        CHECK(grid == tiles * a.splits);
    }
    CHECK((int64_t)d.block_m * a.a_pitch < (int64_t)1 << 31);
    CHECK((a.splits > 1) == (a.partial != nullptr) && a.splits <= GEMM_F16_MAX_SPLITS);
    CHECK((int64_t)a.splits * a.k_split >= a.K && (a.K == 0 || (int64_t)(a.splits - 1) * a.k_split < a.K));
    CHECK(a.splits == 1 || (a.k_split % step == 0 && (int64_t)d.block_m * a.N * 4 < (int64_t)1 << 31));
    return hipSuccess;
}
hipError_t launch_i8_experts(int config, const I8Args &a, int64_t grid, hipStream_t)
{
    check_args(config, a, grid);
    CHECK(a.order && a.starts && a.experts > 0 && a.pairs > 0 && a.pairs_per_row > 0 && a.splits == 1 && !a.partial && a.k_split >= a.K);
    CHECK((int64_t)a.M * a.pairs_per_row == a.pairs && (int64_t)a.M * a.a_pitch < (int64_t)1 << 31);
    const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
    CHECK(a.tiles_m <= a.pairs);
    if (kI8Configs[config].block_m == 256 && kI8Configs[config].block_n == 256)
        CHECK(a.uncut >= tiles && a.uncut % 8 == 0 && grid - a.uncut >= 4 * std::min<int64_t>(tiles, kI8Cut) && (grid - a.uncut) % 32 == 0);
    else
        CHECK(grid == tiles);
    // loads of experts and none, one pair in every tile but one of them, fit the grid
    const int64_t bins = std::min<int64_t>(a.pairs, a.experts + 1), rows = kI8Configs[config].block_m;
    CHECK(bins - 1 + (a.pairs - (bins - 1) + rows - 1) / rows <= a.tiles_m);
    return hipSuccess;
}
hipError_t launch_i8_reduce(const I8Args &a, hipStream_t)
{
    CHECK(a.partial && a.splits > 1 && a.M > 0 && a.N > 0);
    return hipSuccess;
}
hipError_t launch_i8_compress(const _Float16 *X, int64_t stride, int8_t *codes, int64_t pitch, float *scales, int64_t rows, int64_t K,
                              hipStream_t)
{
    ++g_launches;
    CHECK(rows > 0 && K >= 0 && scales && (K == 0 || (X && codes && (uintptr_t)codes % 16 == 0)) && stride >= K);
    CHECK(pitch >= K && pitch % 16 == 0 && pitch == gemm_f16_i8_pitch(K));
    return hipSuccess;
}
hipError_t launch_i8_expand(const int8_t *codes, int64_t pitch, const float *scales, _Float16 *X, int64_t rows, int64_t K, hipStream_t)
{
    ++g_launches;
    CHECK(rows > 0 && K > 0 && X && codes && scales && pitch % 16 == 0 && pitch >= (K + 15) / 16 * 16);
    return hipSuccess;
}
hipError_t launch_route(const RouteArgs &a, hipStream_t)
{
    ++g_launches;
    CHECK(a.logits && a.ids && a.weights && a.tokens > 0 && a.experts > 0 && a.top_k > 0 && a.top_k <= a.experts && a.top_k <= 64);
    CHECK(a.stride >= a.experts && a.experts % a.groups == 0 && a.groups <= 64 && a.top_groups > 0 && a.top_groups <= a.groups);
    CHECK(a.experts <= 1024 && ((int64_t)a.tokens + 3) / 4 * 256 <= 0xffffffff);
    return hipSuccess;
}
hipError_t launch_expert_order(const int32_t *ids, int32_t *order, int32_t *starts, int pairs, int experts, hipStream_t)
{
    ++g_launches;
    CHECK(starts && experts > 0 && experts <= 1024 && pairs >= 0 && (pairs == 0 || (ids && order)) && pairs < 1 << 25);
    return hipSuccess;
}
hipError_t launch_expert_sum(const _Float16 *Y, const float *weights, _Float16 *out, int64_t tokens, int top_k, int64_t N, hipStream_t)
{
    ++g_launches;
    CHECK(out && tokens > 0 && N > 0 && top_k >= 0 && (top_k == 0 || (Y && weights)));
    return hipSuccess;
}
} // namespace gemm_f16_impl

static uint64_t g_rng = 0x9E3779B97F4A7C15ull;
static uint64_t next()
{
    g_rng ^= g_rng << 13;
    g_rng ^= g_rng >> 7;
    g_rng ^= g_rng << 17;
    return g_rng;
}
static int64_t pick(int64_t most)
{
    static const int64_t edges[] = {0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 256, 4100, 8192, 28672, 131071, 131072,
                                    (int64_t)1 << 20, ((int64_t)1 << 20) + 1, ((int64_t)1 << 22) + 1, ((int64_t)1 << 25) - 1,
                                    (int64_t)1 << 25, ((int64_t)1 << 31) - 1, (int64_t)1 << 31, -1};
    return next() % 8 == 0 ? edges[next() % (sizeof(edges) / sizeof(edges[0]))] : (int64_t)(next() % (uint64_t)most);
}
static void *at(int i)
{
    const uint64_t odd[] = {0, 0, 0, 0, 0, 0, 0, 0, 2, 4, 8, 1};
    return next() % 60 == 0 ? nullptr : (void *)(((uint64_t)(i + 1) << 48) + odd[next() % 12]);
}
static int64_t pitch(int64_t k) { return next() % 12 ? (k + 15) / 16 * 16 + 16 * (int64_t)(next() % 3) : pick(10000); }

int main()
{
    int ok = 0;
    for (int i = 0; i < 400000; ++i) {
        const int before = g_launches, kind = (int)(next() % 6), config = (int)(next() % 14) - 1;
        gemm_f16_status_t st;
        bool nothing = false;
        if (kind == 0) {
            const int64_t M = pick(5000), N = pick(9000), K = pick(20000), ap = pitch(K), wp = pitch(K);
            const int splits = next() % 3 ? 0 : (int)(next() % 70) - 1;
            void *ws = next() % 4 ? at(5) : nullptr;
            st = gemm_f16_i8(M, N, K, at(0), ap, (const float *)at(1), at(2), wp, (const float *)at(3), at(4), 0.5f, (int)(next() % 7 % 3),
                             config, splits, ws, ws ? (int64_t)(next() % ((uint64_t)1 << 40)) : 0, nullptr);
            if (st == GEMM_F16_SUCCESS) {
                gemm_f16_plan_t p, again;
                CHECK(gemm_f16_plan_i8(M, N, K, config, splits, &p) == GEMM_F16_SUCCESS);
                CHECK(p.splits >= 1 && p.lds_bytes <= 163840 && (p.workspace_bytes > 0) == (p.splits > 1 && M > 0 && N > 0));
                CHECK(gemm_f16_plan_i8(M, N, K, config, splits, &again) == GEMM_F16_SUCCESS && memcmp(&p, &again, sizeof(p)) == 0);
            }
            nothing = M == 0 || N == 0;
        } else if (kind == 1) {
            const int64_t rows = pick(5000), K = pick(9000);
            const bool compress = next() % 2;
            st = compress ? gemm_f16_i8_compress(rows, K, at(0), K + pick(100), at(1), (float *)at(2), nullptr)
                          : gemm_f16_i8_expand(rows, K, at(1), pitch(K), (const float *)at(2), at(0), nullptr);
            nothing = rows == 0 || (!compress && K == 0);
        } else if (kind == 2) {
            const int64_t tokens = pick(5000), experts = next() % 3 ? 8 << next() % 6 : pick(1100);
            const int groups = next() % 2 ? 1 : 1 << next() % 7;
            st = gemm_f16_route(tokens, (int)experts, (int)pick(12), at(0), (int)(next() % 9 ? next() % 2 : 2), experts + pick(100),
                                (int)(next() % 2), (const float *)(next() % 2 ? at(3) : nullptr), groups, 1 + (int)(next() % groups),
                                (int)(next() % 2), 1.0f, (int32_t *)at(1), (float *)at(2), nullptr);
            nothing = tokens == 0;
        } else if (kind == 3) {
            st = gemm_f16_expert_order(pick(100000), (int)pick(1100), (const int32_t *)at(0), (int32_t *)at(1), (int32_t *)at(2), nullptr);
        } else if (kind == 4) {
            const int64_t per = next() % 10 ? 1 + (int64_t)(next() % 10) : pick(20), pairs = next() % 20 ? per * pick(5000) : pick(50000);
            const int64_t N = pick(9000), K = pick(9000);
            st = gemm_f16_i8_experts(pairs, per, (int)pick(300), N, K, at(0), pitch(K), (const float *)at(1), at(2), pitch(K),
                                     (const float *)at(3), (const int32_t *)at(5), (const int32_t *)at(6), at(4), 0.5f, (int)(next() % 2),
                                     config, nullptr);
            nothing = pairs == 0 || N == 0;
        } else {
            const int64_t tokens = pick(5000), N = pick(9000);
            st = gemm_f16_expert_sum(tokens, pick(20), N, at(0), (const float *)at(1), at(2), nullptr);
            nothing = tokens == 0 || N == 0;
        }
        CHECK(g_launches - before == (st == GEMM_F16_SUCCESS && !nothing ? 1 : 0));
        ok += st == GEMM_F16_SUCCESS;
    }
    printf("%d accepted, %d launches, %d failed checks\n", ok, g_launches, g_fails);
    return g_fails != 0 || ok < 60000;
}
