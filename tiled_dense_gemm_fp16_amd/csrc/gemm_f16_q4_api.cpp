// gemm_f16_q4_api.cpp -- the C ABI of the products with 4-bit operands:
// argument validation, choice of kernel and launch.  Validation and planning
// make no HIP call.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "gemm_f16_internal.h"
#include "gemm_f16_q4.h"
#include "gemm_f16_q4_format.h"

namespace gemm_f16_impl {
namespace {

bool known_group(int group) { return group == 32 || group == 64 || group == 128; }

gemm_f16_status_t status_of(hipError_t e) { return e == hipSuccess ? GEMM_F16_SUCCESS : GEMM_F16_ERROR_LAUNCH_FAILED; }

// W's dimensions and its two buffers
gemm_f16_status_t validate_weights(int64_t N, int64_t K, int group, const void *codes, const void *words)
{
    if (N < 0 || K < 0 || !known_group(group))
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (N > GEMM_F16_MAX_N || K > GEMM_F16_MAX_K)
        return GEMM_F16_ERROR_UNSUPPORTED_SIZE;
    if (N > 0 && K > 0 && (!codes || !words))
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (((uintptr_t)codes | (uintptr_t)words) % 16)
        return GEMM_F16_ERROR_MISALIGNED;
    return GEMM_F16_SUCCESS;
}

gemm_f16_status_t make_plan(int64_t M, int64_t N, int64_t K, int group, int config, gemm_f16_plan_t *p)
{
    if (config != GEMM_F16_CONFIG_AUTO && (config < 0 || config >= kNumQ4Configs))
        return GEMM_F16_ERROR_INVALID_VALUE;
    const int c = config != GEMM_F16_CONFIG_AUTO ? config : M <= 16 ? 0 : M <= 32 ? 1 : 2;
    const Q4Config &d = kQ4Configs[c];
    memset(p, 0, sizeof(*p));
    p->config = c;
    p->block_m = 16 * d.m_blocks;
    p->block_n = 16 * d.n_blocks;
    p->block_k = 128;
    p->stages = 1;
    p->threads = 64 * d.waves;
    p->vec_a = 8;
    p->vec_b = 32;
    p->vec_c = 1;
    p->tiles_m = (M + p->block_m - 1) / p->block_m;
    p->tiles_n = (N + p->block_n - 1) / p->block_n;
    p->grid = p->tiles_m * p->tiles_n;
    p->k_tiles = (K + 127) / 128;
    p->lds_bytes = M > 0 ? q4_lds_bytes(d, M, q4_chunk(d, M, K)) : 0;
    p->flops = 2.0 * (double)M * (double)N * (double)K;
    p->min_bytes = 0.5 * (double)N * (double)K + 4.0 * (double)N * (double)((K + group - 1) / group) +
                   2.0 * (double)M * ((double)N + (double)K);
    p->trans_b = 1;
    p->splits = 1;
    p->k_split = K;
    return GEMM_F16_SUCCESS;
}

} // namespace
} // namespace gemm_f16_impl

using namespace gemm_f16_impl;

extern "C" {

int64_t gemm_f16_q4_codes_bytes(int64_t N, int64_t K)
{
    if (N < 0 || K < 0 || N > GEMM_F16_MAX_N || K > GEMM_F16_MAX_K)
        return -1;
    return (N + 15) / 16 * ((K + 127) / 128) * 1024;
}

int64_t gemm_f16_q4_words_bytes(int64_t N, int64_t K, int group)
{
    if (N < 0 || K < 0 || N > GEMM_F16_MAX_N || K > GEMM_F16_MAX_K || !known_group(group))
        return -1;
    return (N + 15) / 16 * ((K + 127) / 128) * 16 * (128 / group) * 4;
}

gemm_f16_status_t gemm_f16_q4_compress(int64_t N, int64_t K, int group, int symmetric, const void *W, void *codes,
                                       void *words, void *stream)
{
    gemm_f16_status_t st = validate_weights(N, K, group, codes, words);
    if (st != GEMM_F16_SUCCESS)
        return st;
    if (symmetric != 0 && symmetric != 1)
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (N == 0 || K == 0)
        return GEMM_F16_SUCCESS;
    if (!W)
        return GEMM_F16_ERROR_INVALID_VALUE;
    if ((uintptr_t)W & 1u)
        return GEMM_F16_ERROR_MISALIGNED;
    const int64_t cb = gemm_f16_q4_codes_bytes(N, K), wb = gemm_f16_q4_words_bytes(N, K, group);
    if (overlaps(codes, cb, W, 2 * N * K) || overlaps(words, wb, W, 2 * N * K) || overlaps(codes, cb, words, wb))
        return GEMM_F16_ERROR_INVALID_VALUE;
    int dev = -1;
    st = check_device(&dev);
    if (st != GEMM_F16_SUCCESS)
        return st;
    return status_of(launch_q4_compress((const _Float16 *)W, (uint32_t *)codes, (uint32_t *)words, N, K, group,
                                        symmetric != 0, K % 8 == 0 && (uintptr_t)W % 16 == 0, (hipStream_t)stream));
}

gemm_f16_status_t gemm_f16_q4_expand(int64_t N, int64_t K, int group, const void *codes, const void *words, void *W,
                                     void *stream)
{
    gemm_f16_status_t st = validate_weights(N, K, group, codes, words);
    if (st != GEMM_F16_SUCCESS)
        return st;
    if (N == 0 || K == 0)
        return GEMM_F16_SUCCESS;
    if (!W)
        return GEMM_F16_ERROR_INVALID_VALUE;
    if ((uintptr_t)W & 1u)
        return GEMM_F16_ERROR_MISALIGNED;
    if (overlaps(codes, gemm_f16_q4_codes_bytes(N, K), W, 2 * N * K) ||
        overlaps(words, gemm_f16_q4_words_bytes(N, K, group), W, 2 * N * K))
        return GEMM_F16_ERROR_INVALID_VALUE;
    int dev = -1;
    st = check_device(&dev);
    if (st != GEMM_F16_SUCCESS)
        return st;
    return status_of(launch_q4_expand((const uint32_t *)codes, (const uint32_t *)words, (_Float16 *)W, N, K, group,
                                      K % 8 == 0 && (uintptr_t)W % 16 == 0, (hipStream_t)stream));
}

gemm_f16_status_t gemm_f16_q4(int64_t M, int64_t N, int64_t K, int group, const void *A, const void *codes,
                              const void *words, void *C, float alpha, int epilogue, int config, void *stream)
{
    gemm_f16_status_t st = validate_weights(N, K, group, codes, words);
    if (st != GEMM_F16_SUCCESS)
        return st;
    if (M < 0 || (epilogue != GEMM_F16_EPILOGUE_NONE && epilogue != GEMM_F16_EPILOGUE_RELU))
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (M > GEMM_F16_MAX_DIM)
        return GEMM_F16_ERROR_UNSUPPORTED_SIZE;
    if ((M > 0 && K > 0 && !A) || (M > 0 && N > 0 && !C))
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (((uintptr_t)A | (uintptr_t)C) & 1u)
        return GEMM_F16_ERROR_MISALIGNED;
    if (overlaps(C, 2 * M * N, A, 2 * M * K) || overlaps(C, 2 * M * N, codes, gemm_f16_q4_codes_bytes(N, K)) ||
        overlaps(C, 2 * M * N, words, gemm_f16_q4_words_bytes(N, K, group)))
        return GEMM_F16_ERROR_INVALID_VALUE;
    gemm_f16_plan_t plan;
    st = make_plan(M, N, K, group, config, &plan);
    if (st != GEMM_F16_SUCCESS)
        return st;
    if (M == 0 || N == 0)
        return GEMM_F16_SUCCESS;
    int dev = -1;
    st = check_device(&dev);
    if (st != GEMM_F16_SUCCESS)
        return st;
    Q4Args a;
    a.A = (const _Float16 *)A;
    a.codes = (const uint32_t *)codes;
    a.words = (const uint32_t *)words;
    a.C = (_Float16 *)C;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.n_blocks = (int)((N + 15) / 16);
    a.k_blocks = (int)((K + 127) / 128);
    a.chunk = q4_chunk(kQ4Configs[plan.config], M, K);
    a.vec_a = K % 8 == 0 && (uintptr_t)A % 16 == 0;
    a.alpha = K == 0 ? 1.0f : alpha;   // the empty sum is +0 whatever alpha
    a.relu = epilogue == GEMM_F16_EPILOGUE_RELU ? 1 : 0;
    return status_of(launch_q4(plan.config, group, a, plan.tiles_n, plan.tiles_m, (hipStream_t)stream));
}

gemm_f16_status_t gemm_f16_plan_q4(int64_t M, int64_t N, int64_t K, int group, int config, gemm_f16_plan_t *plan)
{
    if (!plan || M < 0 || N < 0 || K < 0 || !known_group(group))
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (M > GEMM_F16_MAX_DIM || N > GEMM_F16_MAX_N || K > GEMM_F16_MAX_K)
        return GEMM_F16_ERROR_UNSUPPORTED_SIZE;
    return make_plan(M, N, K, group, config, plan);
}

int gemm_f16_q4_num_configs(void) { return kNumQ4Configs; }

const char *gemm_f16_q4_config_name(int config)
{
    if (config < 0 || config >= kNumQ4Configs)
        return nullptr;
    return kQ4Configs[config].name;
}

} // extern "C"
