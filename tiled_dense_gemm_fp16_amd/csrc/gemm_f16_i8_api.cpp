// gemm_f16_i8_api.cpp -- the C ABI of the products with 8-bit operands and of
// the routed experts: argument validation, choice of kernel and launch.
// Validation and planning make no HIP call.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <cmath>

#include "gemm_f16_i8_internal.h"

namespace gemm_f16_impl {

const I8Config kI8Configs[kNumI8Configs] = {
    {"i8_16x16", 16, 16, 8, 0, 4, 1.3f, 2.2f, 1.0f, 4.5f},
    {"i8_32x32_s8", 32, 32, 4, 8, 2, 0.099f, 3.7f, 0.28f, 5.2f},
    {"i8_32x64_s6", 32, 64, 4, 6, 2, 0.156f, 3.7f, 0.17f, 4.2f},
    {"i8_64x64_s6", 64, 64, 8, 6, 1, 0.228f, 3.7f, 0.31f, 3.6f},
    {"i8_64x128_s4", 64, 128, 8, 4, 1, 0.353f, 3.7f, 0.38f, 3.8f},
    {"i8_64x256_s3", 64, 256, 8, 3, 1, 0.542f, 4.6f, 0.71f, 3.6f},
    {"i8_128x128_s4", 128, 128, 8, 4, 1, 0.495f, 4.6f, 0.5f, 4.6f},
    {"i8_128x192_s3", 128, 192, 8, 3, 1, 0.62f, 5.0f, 0.66f, 6.2f},
    {"i8_128x256_s3", 128, 256, 8, 3, 1, 0.766f, 4.9f, 0.74f, 5.2f},
    {"i8_256x128_s3", 256, 128, 4, 3, 1, 0.736f, 6.0f, 0.69f, 6.7f},
    {"i8_256x256_s2", 256, 256, 8, 2, 1, 1.25f, 7.2f, 1.3f, 8.6f},
};

namespace {

constexpr int64_t kMostBytes = (int64_t)1 << 56;   // sizes are refused before their product in 64 bits could overflow

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Work items of a launch's grid are counted in 32 bits.
bool launchable(int64_t workgroups, int64_t threads) { return workgroups <= 0xffffffff / threads; }

gemm_f16_status_t status_of(hipError_t e) { return e == hipSuccess ? GEMM_F16_SUCCESS : GEMM_F16_ERROR_LAUNCH_FAILED; }

int64_t padded(int64_t K) { return (K + 15) / 16 * 16; }

// Rows that compress writes start on cache lines, but the shortest: 1000 x 5000 x
// 4100 with rows of 4112 bytes 39 us, of 4224 28.5 (operands that are still in a
// cache 29, 25); 8192 x 8192 x 4100 247, 220.
int64_t made_pitch(int64_t K) { return K <= 64 ? padded(K) : (K + 127) / 128 * 128; }

// a * b without overflow, beyond kMostBytes where it is more (a, b not negative)
int64_t bytes_of(int64_t a, int64_t b) { return b > 0 && a > kMostBytes / b ? kMostBytes + 1 : a * b; }

// An 8-bit matrix of `rows` rows by K.
gemm_f16_status_t validate_matrix(int64_t rows, int64_t K, const void *codes, int64_t pitch, const float *scales)
{
    if (rows < 0 || K < 0)
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (K > GEMM_F16_I8_MAX_K || pitch > GEMM_F16_MAX_K || rows > GEMM_F16_MAX_DIM)
        return GEMM_F16_ERROR_UNSUPPORTED_SIZE;
    if (pitch < padded(K) || pitch % 16 != 0)
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (rows > 0 && ((K > 0 && !codes) || !scales))
        return GEMM_F16_ERROR_INVALID_VALUE;
    if ((uintptr_t)codes % 16 || (uintptr_t)scales % 4)
        return GEMM_F16_ERROR_MISALIGNED;
    return GEMM_F16_SUCCESS;
}

int vec_of(const void *C, int64_t N)
{
    return N % 8 == 0 && (uintptr_t)C % 16 == 0 ? 8 : N % 4 == 0 && (uintptr_t)C % 8 == 0 ? 4 : 1;
}

// Elements that a store of a 16-byte aligned C takes, for a plan: a split's sum
// stores four at most, and the kernel for few rows one at a time.
int planned_vec_c(const I8Config &d, int64_t N, int splits)
{
    const int most = splits > 1 ? 4 : d.stages > 0 ? 8 : 1;
    return std::min(vec_of(nullptr, N), most);
}

void describe(int c, bool experts, gemm_f16_plan_t *p)
{
    const I8Config &d = kI8Configs[c];
    memset(p, 0, sizeof(*p));
    p->config = c;
    p->block_m = d.block_m;
    p->block_n = d.block_n;
    p->block_k = d.stages > 0 ? kI8BlockK : kI8StreamK;
    p->stages = d.stages > 0 ? d.stages : 1;
    p->threads = 64 * d.waves;
    p->direct_lds = d.stages > 0;
    p->vec_a = p->vec_b = 16;
    p->trans_b = 1;
    p->lds_bytes = d.stages > 0 ? i8_lds_bytes(d.block_m, d.block_n, d.stages, experts) : d.waves * d.block_n * 64;
}

// Whether a configuration's last round may be cut into quarters of its tiles,
// and the workgroups for those (eight tiles at a time, one for each XCD).
bool cuts(const I8Config &d) { return d.block_m == 256 && d.block_n == 256; }
int64_t quarters(int64_t tiles) { return 4 * 8 * ceil_div(tiles, 8); }

// A product's time in us, for the choice of a configuration and split: rounds of
// workgroups over 256 CUs, or the time to bring W from memory and the tiles'
// operands from the L2s if that is longer, and a split's partial sums and second
// launch.  The configurations' constants and the rates below were fitted to what
// 731 shapes (M 1 to 4096, N 256 to 28672, K 512 to 16384) took in every
// configuration and split, not for the times but so that the choice comes out
// right: it took 2 % longer than the best one on average, a quarter at most but for
// a few shapes.  (The kernel for few rows keeps a CU's loads busy by itself, so
// where some CUs have two of its workgroups and the others one, it is half as fast:
// (16, 5000 x 4096) 11.6 us, 32x32 9.3.)  us of some choices and others, weights from
// memory: (1, 28672 x 8192) 16x16 43, 32x64 52; (1000, 5000 x 4096) 128x192 28, 128x256
// 31, 256x128 32, 128x128 41, 256x256 42; (8192, 8192 x 8192) 256x256 420, 256x128 459,
// 128x256 464, 128x128 570.  Where the choice depends on whether the weights are still
// in a cache, it is the best one if they are: (64, 8192 x 8192) 32x64 14.3, 64x128 in 4
// parts 17.7, but from memory 23 and 21; (32, 8192 x 8192) 32x64 14.1, from memory 24
// (32x32 19).
double estimate(const I8Config &d, int64_t M, int64_t N, int64_t K, int splits)
{
    const int64_t tiles = ceil_div(M, d.block_m) * ceil_div(N, d.block_n) * splits;
    const int64_t step_k = d.stages > 0 ? kI8BlockK : 8 * kI8StreamK;
    const double fixed = d.fixed, steps = (double)ceil_div(ceil_div(K, splits), step_k);
    double rounds = (double)ceil_div(tiles, 256 * d.resident);
    if (cuts(d) && splits == 1 && tiles % 256 > 0 && tiles % 256 <= kI8Cut)
        rounds += (tiles % 256 <= kI8Cut / 2 ? 0.45 : 0.9) - 1.0;   // one or two rounds of quarters
    if (d.stages == 0 && tiles > 256 && tiles < 448)
        rounds = 1.5;
    const double memory = ((double)N * K + 2.0 * M * N) / 16e6 +
                          (double)tiles * ceil_div(K, splits) * (double)(std::min<int64_t>(d.block_m, M) + d.block_n) / 20e6;
    return std::max(rounds * (fixed + steps * d.step), fixed + memory) + (splits > 1 ? 2.7 + 8.0 * M * N * splits / 5.2e6 : 0.0);
}

// The same over experts, of which only the number of pairs is known here: as
// many experts as may be have an equal share, in tiles of which the last is half
// full, and an uneven load fills a quarter of a round more.  Fitted to 186 loads (8 to
// 256 experts, 1 to 4096 tokens, 2 or 8 experts each, some experts more popular): 2 %
// longer than the best on average.  us: 64 tokens, 8 of 256 experts of 4096 x 2048
// 64x256 254, 32x64 326, 128x128 291; 2048 tokens, 8 of 64 of 2048 x 4096 256x256
// 197 to 206, 128x256 200, 128x128 254; 1 token, 8 of 256 of 2048 x 4096 32x64 15.1,
// 64x256 19.6.
double estimate_experts(const I8Config &d, int64_t pairs, int experts, int64_t N, int64_t K)
{
    const double hit = (double)std::min<int64_t>(experts, pairs), rows = (double)pairs / hit;
    const double tiles = hit * std::max(1.0, rows / d.block_m + 0.5) * (double)ceil_div(N, d.block_n);
    const double fixed = d.experts_fixed, steps = (double)ceil_div(K, d.stages > 0 ? kI8BlockK : 8 * kI8StreamK);
    const double memory = (hit * (double)N * (double)K + 2.0 * (double)pairs * (double)N) / 12e6 +
                          tiles * (double)K * (std::min((double)d.block_m, rows) + d.block_n) / 14e6;
    return std::max(std::max(1.0, tiles / (256.0 * d.resident) + 0.25) * (fixed + steps * d.experts_step), fixed + memory);
}

// Choices that this thread made last, so that a program that repeats its shapes
// does not search again (0.7 us).
struct Choice {
    int64_t key[5] = {-1, -1, -1, -1, -1};
    int config = 0, splits = 0;
};
Choice &remembered(const int64_t (&key)[5])
{
    static thread_local Choice choices[64];
    uint64_t h = 0;
    for (int64_t k : key)
        h = (h ^ (uint64_t)k) * 0x9e3779b97f4a7c15ull;
    return choices[h >> 58];
}
bool same(const int64_t (&a)[5], const int64_t (&b)[5]) { return std::equal(a, a + 5, b); }

// Splits of an automatic plan: parts of 4 steps and more that make no more
// than two workgroups for each CU.
constexpr int kSplits[] = {1, 2, 4, 8};
bool may_split(const I8Config &d, int64_t M, int64_t N, int64_t K, int splits)
{
    const int64_t tiles = ceil_div(M, d.block_m) * ceil_div(N, d.block_n);
    return splits == 1 || (tiles < 256 && tiles * splits <= 512 && N <= (int64_t)1 << 20 &&
                           ceil_div(K, d.stages > 0 ? kI8BlockK : kI8StreamK) >= 4 * splits);
}

gemm_f16_status_t plan_product(int64_t M, int64_t N, int64_t K, int config, int splits, gemm_f16_plan_t *p)
{
    if (M < 0 || N < 0 || K < 0 || (config != GEMM_F16_CONFIG_AUTO && (config < 0 || config >= kNumI8Configs)) || splits < 0 ||
        splits > GEMM_F16_MAX_SPLITS)
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (M > GEMM_F16_MAX_DIM || N > GEMM_F16_MAX_N || K > GEMM_F16_I8_MAX_K)
        return GEMM_F16_ERROR_UNSUPPORTED_SIZE;
    int c = config == GEMM_F16_CONFIG_AUTO ? 0 : config;
    const int64_t key[5] = {M, N, K, config, splits};
    Choice &last = remembered(key);
    if (same(last.key, key)) {
        c = last.config;
        splits = last.splits;
    } else if (config == GEMM_F16_CONFIG_AUTO || splits == GEMM_F16_SPLITS_AUTO) {
        double best = HUGE_VAL;
        int request = std::max(splits, 1);
        for (int i = 0; i < kNumI8Configs; ++i) {
            if ((config != GEMM_F16_CONFIG_AUTO && i != config) || (config == GEMM_F16_CONFIG_AUTO && i == 0 && M > 16))
                continue;
            const int64_t tiles = ceil_div(M, kI8Configs[i].block_m) * ceil_div(N, kI8Configs[i].block_n);
            if (config == GEMM_F16_CONFIG_AUTO && !launchable(tiles * std::max(splits, 1), 64 * kI8Configs[i].waves))
                continue;
            for (int s : kSplits) {
                if (splits != GEMM_F16_SPLITS_AUTO)
                    s = splits;
                else if (!may_split(kI8Configs[i], M, N, K, s))
                    continue;
                const double t = estimate(kI8Configs[i], M, N, K, s);
                if (t < best) {
                    best = t;
                    c = i;
                    request = s;
                }
            }
        }
        splits = request;
        std::copy(key, key + 5, last.key);
        last.config = c;
        last.splits = splits;
    }
    const I8Config &d = kI8Configs[c];
    describe(c, false, p);
    p->flops = 2.0 * (double)M * (double)N * (double)K;
    p->min_bytes = ((double)M + (double)N) * ((double)K + 4.0) + 2.0 * (double)M * (double)N;
    p->tiles_m = ceil_div(M, d.block_m);
    p->tiles_n = ceil_div(N, d.block_n);
    const int64_t tiles = p->tiles_m * p->tiles_n, steps = ceil_div(K, p->block_k);
    const int64_t per = steps > 0 ? ceil_div(steps, splits) : 0;
    p->splits = per > 0 ? (int)ceil_div(steps, per) : 1;   // none empty
    // (a split's sums of a tile's rows are reached by offsets of 31 bits)
    if (p->splits > 1 && N > (int64_t)1 << 20)
        return GEMM_F16_ERROR_UNSUPPORTED_SIZE;
    p->k_tiles = per;
    p->k_split = p->splits > 1 ? per * p->block_k : K;
    p->grid = cuts(d) && p->splits == 1 && tiles <= INT32_MAX ? i8_uncut((int)tiles) + quarters(tiles - i8_uncut((int)tiles))
                                                              : tiles * p->splits;
    p->workspace_bytes = p->splits > 1 ? (int64_t)p->splits * M * N * 4 : 0;
    p->vec_c = planned_vec_c(d, N, p->splits);
    return launchable(p->grid, p->threads) ? GEMM_F16_SUCCESS : GEMM_F16_ERROR_UNSUPPORTED_SIZE;
}

// Tiles of `rows` pairs at most: each expert's last one, and that of the pairs of none, may hold one pair.
int64_t most_tiles(int64_t pairs, int experts, int rows)
{
    return std::min<int64_t>(pairs, (pairs + std::min<int64_t>(pairs, experts + 1) * (rows - 1)) / rows);
}

gemm_f16_status_t plan_experts(int64_t pairs, int64_t per_row, int experts, int64_t N, int64_t K, int config, gemm_f16_plan_t *p)
{
    if (pairs < 0 || per_row < 1 || pairs % per_row != 0 || experts < 1 || N < 0 || K < 0 ||
        (config != GEMM_F16_CONFIG_AUTO && (config < 0 || config >= kNumI8Configs)))
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (pairs > GEMM_F16_MAX_PAIRS || experts > GEMM_F16_MAX_EXPERTS || N > GEMM_F16_MAX_N || K > GEMM_F16_I8_MAX_K)
        return GEMM_F16_ERROR_UNSUPPORTED_SIZE;
    int c = config == GEMM_F16_CONFIG_AUTO ? 0 : config;
    const int64_t key[5] = {pairs, N, K, experts, -2};   // (no product's)
    Choice &last = remembered(key);
    if (config == GEMM_F16_CONFIG_AUTO && same(last.key, key)) {
        c = last.config;
    } else if (config == GEMM_F16_CONFIG_AUTO && pairs > 0) {
        double best = HUGE_VAL;
        for (int i = 0; i < kNumI8Configs; ++i) {
            const I8Config &d = kI8Configs[i];
            if ((i == 0 && pairs > 16 * (int64_t)experts) ||
                !launchable(most_tiles(pairs, experts, d.block_m) * ceil_div(N, d.block_n), 64 * d.waves))
                continue;
            const double t = estimate_experts(kI8Configs[i], pairs, experts, N, K);
            if (t < best) {
                best = t;
                c = i;
            }
        }
        std::copy(key, key + 5, last.key);
        last.config = c;
    }
    const I8Config &d = kI8Configs[c];
    describe(c, true, p);
    p->splits = 1;
    p->vec_c = planned_vec_c(d, N, 1);
    p->k_split = K;
    p->k_tiles = ceil_div(K, p->block_k);
    p->flops = 2.0 * (double)pairs * (double)N * (double)K;
    p->min_bytes = ((double)experts * (double)N + (double)(pairs / per_row)) * ((double)K + 4.0) + 2.0 * (double)pairs * (double)N;
    p->tiles_m = most_tiles(pairs, experts, d.block_m);
    p->tiles_n = ceil_div(N, d.block_n);
    const int64_t tiles = p->tiles_m * p->tiles_n;
    p->grid = cuts(d) ? ceil_div(tiles, 8) * 8 + quarters(std::min<int64_t>(tiles, kI8Cut)) : tiles;
    return launchable(p->grid, p->threads) ? GEMM_F16_SUCCESS : GEMM_F16_ERROR_UNSUPPORTED_SIZE;
}

I8Args arguments(const void *A, int64_t a_pitch, const float *a_scales, const void *W, int64_t w_pitch, const float *w_scales,
                 void *C, int64_t N, int64_t K, float alpha, int epilogue, const gemm_f16_plan_t &plan)
{
    I8Args a;
    memset(&a, 0, sizeof(a));
    a.A = (const int8_t *)A;
    a.W = (const int8_t *)W;
    a.a_scales = a_scales;
    a.w_scales = w_scales;
    a.C = (_Float16 *)C;
    a.a_pitch = a_pitch;
    a.w_pitch = w_pitch;
    a.N = (int)N;
    a.K = (int)padded(K);
    a.tiles_m = (int)plan.tiles_m;
    a.tiles_n = (int)plan.tiles_n;
    a.splits = plan.splits;
    a.k_split = plan.splits > 1 ? (int)plan.k_split : a.K;
    a.alpha = alpha;
    a.relu = epilogue == GEMM_F16_EPILOGUE_RELU ? 1 : 0;
    a.vec_c = vec_of(C, N);
    return a;
}

bool known_epilogue(int e) { return e == GEMM_F16_EPILOGUE_NONE || e == GEMM_F16_EPILOGUE_RELU; }

} // namespace
} // namespace gemm_f16_impl

using namespace gemm_f16_impl;

extern "C" {

int64_t gemm_f16_i8_pitch(int64_t K) { return K < 0 || K > GEMM_F16_I8_MAX_K ? -1 : made_pitch(K); }

gemm_f16_status_t gemm_f16_i8_compress(int64_t rows, int64_t K, const void *X, int64_t x_stride, void *codes, float *scales,
                                       void *stream)
{
    gemm_f16_status_t st = validate_matrix(rows, K, codes, gemm_f16_i8_pitch(K < 0 ? 0 : std::min(K, GEMM_F16_I8_MAX_K)), scales);
    if (st != GEMM_F16_SUCCESS)
        return st;
    if (rows == 0)
        return GEMM_F16_SUCCESS;
    if ((K > 0 && !X) || x_stride < K)
        return GEMM_F16_ERROR_INVALID_VALUE;
    if ((uintptr_t)X & 1u)
        return GEMM_F16_ERROR_MISALIGNED;
    if (bytes_of(rows, x_stride) > kMostBytes / 2)
        return GEMM_F16_ERROR_UNSUPPORTED_SIZE;
    const int64_t x_bytes = 2 * ((rows - 1) * x_stride + K), pitch = made_pitch(K), c_bytes = rows * pitch;
    if (overlaps(codes, c_bytes, X, x_bytes) || overlaps(scales, 4 * rows, X, x_bytes) || overlaps(codes, c_bytes, scales, 4 * rows))
        return GEMM_F16_ERROR_INVALID_VALUE;
    int dev = -1;
    st = check_device(&dev);
    if (st != GEMM_F16_SUCCESS)
        return st;
    return status_of(launch_i8_compress((const _Float16 *)X, x_stride, (int8_t *)codes, pitch, scales, rows, K, (hipStream_t)stream));
}

gemm_f16_status_t gemm_f16_i8_expand(int64_t rows, int64_t K, const void *codes, int64_t pitch, const float *scales, void *X,
                                     void *stream)
{
    gemm_f16_status_t st = validate_matrix(rows, K, codes, pitch, scales);
    if (st != GEMM_F16_SUCCESS)
        return st;
    if (rows == 0 || K == 0)
        return GEMM_F16_SUCCESS;
    if (!X)
        return GEMM_F16_ERROR_INVALID_VALUE;
    if ((uintptr_t)X & 1u)
        return GEMM_F16_ERROR_MISALIGNED;
    const int64_t x_bytes = 2 * rows * K;
    if (overlaps(X, x_bytes, codes, rows * pitch) || overlaps(X, x_bytes, scales, 4 * rows))
        return GEMM_F16_ERROR_INVALID_VALUE;
    int dev = -1;
    st = check_device(&dev);
    if (st != GEMM_F16_SUCCESS)
        return st;
    return status_of(launch_i8_expand((const int8_t *)codes, pitch, scales, (_Float16 *)X, rows, K, (hipStream_t)stream));
}

gemm_f16_status_t gemm_f16_i8(int64_t M, int64_t N, int64_t K, const void *A, int64_t a_pitch, const float *a_scales,
                              const void *W, int64_t w_pitch, const float *w_scales, void *C, float alpha, int epilogue,
                              int config, int splits, void *workspace, int64_t workspace_bytes, void *stream)
{
    gemm_f16_plan_t plan;
    gemm_f16_status_t st = plan_product(M, N, K, config, splits, &plan);
    if (st != GEMM_F16_SUCCESS)
        return st;
    if (!known_epilogue(epilogue) || workspace_bytes < 0 || (!workspace && workspace_bytes != 0))
        return GEMM_F16_ERROR_INVALID_VALUE;
    st = validate_matrix(M, K, A, a_pitch, a_scales);
    if (st == GEMM_F16_SUCCESS)
        st = validate_matrix(N, K, W, w_pitch, w_scales);
    if (st != GEMM_F16_SUCCESS)
        return st;
    if (M == 0 || N == 0)
        return GEMM_F16_SUCCESS;
    if (!C)
        return GEMM_F16_ERROR_INVALID_VALUE;
    if ((uintptr_t)C & 1u)
        return GEMM_F16_ERROR_MISALIGNED;
    const auto meets_inputs = [&](const void *p, int64_t bytes) {
        return overlaps(p, bytes, A, M * a_pitch) || overlaps(p, bytes, W, N * w_pitch) || overlaps(p, bytes, a_scales, 4 * M) ||
               overlaps(p, bytes, w_scales, 4 * N);
    };
    if (meets_inputs(C, 2 * M * N))
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (plan.splits > 1) {
        if (!workspace)
            return GEMM_F16_ERROR_WORKSPACE;
        if ((uintptr_t)workspace % 16)
            return GEMM_F16_ERROR_MISALIGNED;
        if (workspace_bytes < plan.workspace_bytes)
            return GEMM_F16_ERROR_WORKSPACE;
        if (meets_inputs(workspace, plan.workspace_bytes) || overlaps(workspace, plan.workspace_bytes, C, 2 * M * N))
            return GEMM_F16_ERROR_INVALID_VALUE;
    }
    int dev = -1;
    st = check_device(&dev);
    if (st != GEMM_F16_SUCCESS)
        return st;
    I8Args a = arguments(A, a_pitch, a_scales, W, w_pitch, w_scales, C, N, K, alpha, epilogue, plan);
    a.M = (int)M;
    a.partial = plan.splits > 1 ? (int *)workspace : nullptr;
    if (cuts(kI8Configs[plan.config]))
        a.uncut = i8_uncut(a.tiles_m * a.tiles_n);
    const hipError_t e = launch_i8(plan.config, a, plan.grid, (hipStream_t)stream);
    if (e != hipSuccess || plan.splits == 1)
        return status_of(e);
    return status_of(launch_i8_reduce(a, (hipStream_t)stream));
}

gemm_f16_status_t gemm_f16_plan_i8(int64_t M, int64_t N, int64_t K, int config, int splits, gemm_f16_plan_t *plan)
{
    if (!plan)
        return GEMM_F16_ERROR_INVALID_VALUE;
    return plan_product(M, N, K, config, splits, plan);
}

int gemm_f16_i8_num_configs(void) { return kNumI8Configs; }

const char *gemm_f16_i8_config_name(int config)
{
    if (config < 0 || config >= kNumI8Configs)
        return nullptr;
    return kI8Configs[config].name;
}

gemm_f16_status_t gemm_f16_route(int64_t tokens, int experts, int top_k, const void *logits, int half, int64_t stride, int score,
                                 const float *bias, int groups, int top_groups, int renormalise, float scale, int32_t *ids,
                                 float *weights, void *stream)
{
    if (tokens < 0 || experts < 1 || top_k < 1 || top_k > experts || (half != 0 && half != 1) ||
        (score != GEMM_F16_SCORE_SOFTMAX && score != GEMM_F16_SCORE_SIGMOID) || groups < 1 || experts % groups != 0 ||
        top_groups < 1 || top_groups > groups || (renormalise != 0 && renormalise != 1) || !std::isfinite(scale))
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (experts > GEMM_F16_MAX_EXPERTS || top_k > GEMM_F16_MAX_TOP_K || groups > GEMM_F16_MAX_EXPERT_GROUPS ||
        tokens > GEMM_F16_MAX_PAIRS / top_k)
        return GEMM_F16_ERROR_UNSUPPORTED_SIZE;
    if (tokens == 0)
        return GEMM_F16_SUCCESS;
    if (!logits || !ids || !weights || stride < experts)
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (bytes_of(tokens, stride) > kMostBytes / 4)
        return GEMM_F16_ERROR_UNSUPPORTED_SIZE;
    if ((uintptr_t)logits % (half ? 2 : 4) || ((uintptr_t)ids | (uintptr_t)weights | (uintptr_t)bias) % 4)
        return GEMM_F16_ERROR_MISALIGNED;
    const int64_t in = ((tokens - 1) * stride + experts) * (half ? 2 : 4), out = 4 * tokens * top_k;
    if (overlaps(ids, out, weights, out) || overlaps(ids, out, logits, in) || overlaps(weights, out, logits, in) ||
        (bias && (overlaps(ids, out, bias, 4 * experts) || overlaps(weights, out, bias, 4 * experts))))
        return GEMM_F16_ERROR_INVALID_VALUE;
    int dev = -1;
    const gemm_f16_status_t st = check_device(&dev);
    if (st != GEMM_F16_SUCCESS)
        return st;
    RouteArgs a;
    a.logits = logits;
    a.bias = bias;
    a.ids = ids;
    a.weights = weights;
    a.stride = stride;
    a.tokens = (int)tokens;
    a.experts = experts;
    a.top_k = top_k;
    a.half = half;
    a.sigmoid = score == GEMM_F16_SCORE_SIGMOID;
    a.groups = groups;
    a.top_groups = top_groups;
    a.renormalise = renormalise;
    a.scale = scale;
    return status_of(launch_route(a, (hipStream_t)stream));
}

gemm_f16_status_t gemm_f16_expert_order(int64_t pairs, int experts, const int32_t *ids, int32_t *order, int32_t *starts,
                                        void *stream)
{
    if (pairs < 0 || experts < 1)
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (pairs > GEMM_F16_MAX_PAIRS || experts > GEMM_F16_MAX_EXPERTS)
        return GEMM_F16_ERROR_UNSUPPORTED_SIZE;
    if (!starts || (pairs > 0 && (!ids || !order)))
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (((uintptr_t)ids | (uintptr_t)order | (uintptr_t)starts) % 4)
        return GEMM_F16_ERROR_MISALIGNED;
    const int64_t s_bytes = 4 * ((int64_t)experts + 1);
    if (overlaps(order, 4 * pairs, ids, 4 * pairs) || overlaps(order, 4 * pairs, starts, s_bytes) ||
        overlaps(ids, 4 * pairs, starts, s_bytes))
        return GEMM_F16_ERROR_INVALID_VALUE;
    int dev = -1;
    const gemm_f16_status_t st = check_device(&dev);
    if (st != GEMM_F16_SUCCESS)
        return st;
    return status_of(launch_expert_order(ids, order, starts, (int)pairs, experts, (hipStream_t)stream));
}

gemm_f16_status_t gemm_f16_i8_experts(int64_t pairs, int64_t pairs_per_row, int experts, int64_t N, int64_t K, const void *A,
                                      int64_t a_pitch, const float *a_scales, const void *W, int64_t w_pitch,
                                      const float *w_scales, const int32_t *order, const int32_t *starts, void *C, float alpha,
                                      int epilogue, int config, void *stream)
{
    gemm_f16_plan_t plan;
    gemm_f16_status_t st = plan_experts(pairs, pairs_per_row, experts, N, K, config, &plan);
    if (st != GEMM_F16_SUCCESS)
        return st;
    if (!known_epilogue(epilogue))
        return GEMM_F16_ERROR_INVALID_VALUE;
    const int64_t rows = pairs / pairs_per_row, w_rows = (int64_t)experts * N;
    st = validate_matrix(rows, K, A, a_pitch, a_scales);
    if (st == GEMM_F16_SUCCESS)   // (more rows than a product's: 2^32 at most)
        st = validate_matrix(std::min<int64_t>(w_rows, GEMM_F16_MAX_DIM), K, W, w_pitch, w_scales);
    if (st != GEMM_F16_SUCCESS)
        return st;
    if (pairs == 0 || N == 0)
        return GEMM_F16_SUCCESS;
    if (rows * a_pitch > GEMM_F16_MAX_DIM)
        return GEMM_F16_ERROR_UNSUPPORTED_SIZE;
    if (!order || !starts || !C)
        return GEMM_F16_ERROR_INVALID_VALUE;
    if ((uintptr_t)C & 1u || ((uintptr_t)order | (uintptr_t)starts) % 4)
        return GEMM_F16_ERROR_MISALIGNED;
    const int64_t c_bytes = 2 * pairs * N;
    if (overlaps(C, c_bytes, A, rows * a_pitch) || overlaps(C, c_bytes, a_scales, 4 * rows) ||
        overlaps(C, c_bytes, W, w_rows * w_pitch) || overlaps(C, c_bytes, w_scales, 4 * w_rows) ||
        overlaps(C, c_bytes, order, 4 * pairs) || overlaps(C, c_bytes, starts, 4 * ((int64_t)experts + 1)))
        return GEMM_F16_ERROR_INVALID_VALUE;
    int dev = -1;
    st = check_device(&dev);
    if (st != GEMM_F16_SUCCESS)
        return st;
    I8Args a = arguments(A, a_pitch, a_scales, W, w_pitch, w_scales, C, N, K, alpha, epilogue, plan);
    a.M = (int)rows;
    a.order = order;
    a.starts = starts;
    a.experts = experts;
    a.pairs = (int)pairs;
    a.pairs_per_row = (int)pairs_per_row;
    if (cuts(kI8Configs[plan.config]))
        a.uncut = (int)(ceil_div(plan.tiles_m * plan.tiles_n, 8) * 8);
    return status_of(launch_i8_experts(plan.config, a, plan.grid, (hipStream_t)stream));
}

gemm_f16_status_t gemm_f16_plan_i8_experts(int64_t pairs, int64_t pairs_per_row, int experts, int64_t N, int64_t K, int config,
                                           gemm_f16_plan_t *plan)
{
    if (!plan)
        return GEMM_F16_ERROR_INVALID_VALUE;
    return plan_experts(pairs, pairs_per_row, experts, N, K, config, plan);
}

gemm_f16_status_t gemm_f16_expert_sum(int64_t tokens, int64_t top_k, int64_t N, const void *Y, const float *weights, void *out,
                                      void *stream)
{
    if (tokens < 0 || top_k < 0 || N < 0)
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (N > GEMM_F16_MAX_N || top_k > GEMM_F16_MAX_EXPERTS || tokens > GEMM_F16_MAX_PAIRS / std::max<int64_t>(top_k, 1))
        return GEMM_F16_ERROR_UNSUPPORTED_SIZE;
    if (tokens == 0 || N == 0)
        return GEMM_F16_SUCCESS;
    if (!out || (top_k > 0 && (!Y || !weights)))
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (((uintptr_t)Y | (uintptr_t)out) & 1u || (uintptr_t)weights % 4)
        return GEMM_F16_ERROR_MISALIGNED;
    if (overlaps(out, 2 * tokens * N, Y, 2 * tokens * top_k * N) || overlaps(out, 2 * tokens * N, weights, 4 * tokens * top_k))
        return GEMM_F16_ERROR_INVALID_VALUE;
    int dev = -1;
    const gemm_f16_status_t st = check_device(&dev);
    if (st != GEMM_F16_SUCCESS)
        return st;
    return status_of(launch_expert_sum((const _Float16 *)Y, weights, (_Float16 *)out, tokens, (int)top_k, N, (hipStream_t)stream));
}

} // extern "C"
