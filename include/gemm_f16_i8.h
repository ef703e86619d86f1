/*
 * gemm_f16_i8.h -- C ABI of the products with 8-bit operands of the FP16 GEMM
 * library for AMD Instinct MI355X (gfx950), and of layers of routed experts
 * made of them.
 *
 * The pages whose tile GEMM the library implements name mixtures of experts
 * and quantised products among the operators built on the same tiles
 * ("5分钟上手TileLang：GPU内核开发指南", section "进阶方向：从 GEMM 到真实模型算子"),
 * without a format or a definition.  Those here are the library's own.
 *
 * Format.  An 8-bit matrix of `rows` rows by K columns is
 *   codes  : int8, rows of `pitch` bytes, a multiple of 16 that is at least K
 *            rounded up to a multiple of 16; 16-byte aligned.  The codes from K
 *            up to that multiple are zeros.
 *   scales : fp32, one for each row (a token, or an output channel of a
 *            weight matrix); element k of row r stands for scales[r] codes[r][k].
 *
 * Ownership, streams, errors: as in gemm_f16.h.  Buffers belong to the
 * caller, nothing is allocated, nothing synchronises, every entry point may
 * be captured into a HIP graph, and results are bitwise reproducible.
 * Arguments are validated before any HIP call; on error nothing is launched.
 */
#ifndef GEMM_F16_I8_H
#define GEMM_F16_I8_H

#include "gemm_f16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- rows in 8 bits ----------------------------------------------------------
 * Limits: K < 2^17 (sums of products of codes stay within 32 bits), rows <
 * 2^31 (beyond them, and where a buffer would have more than 2^56 bytes:
 * GEMM_F16_ERROR_UNSUPPORTED_SIZE). */
#define GEMM_F16_I8_MAX_K (((int64_t)1 << 17) - 1)

/* The pitch of the rows that gemm_f16_i8_compress writes: K rounded up to a
 * multiple of 16, from 65 on of 128 (whole cache lines); -1 for a K out of range. */
int64_t gemm_f16_i8_pitch(int64_t K);

/*
 * Round rows of X (binary16, x_stride >= K elements apart, 2-byte aligned) to
 * codes (pitch gemm_f16_i8_pitch(K), with zeros from K to the pitch) and scales.  With
 * m = max |x| of the row, NaN counting as 0 and infinities as 65504:
 *   scale = m / 127, rounded to fp32
 *   code  = 127 x / m, rounded to the nearest integer, halves to the even one
 * and both 0 where m = 0.
 */
gemm_f16_status_t gemm_f16_i8_compress(int64_t rows, int64_t K, const void *X, int64_t x_stride, void *codes,
                                       float *scales, void *stream);

/* X = scale code, rounded to fp32 and then to binary16, rows x K row-major, contiguous. */
gemm_f16_status_t gemm_f16_i8_expand(int64_t rows, int64_t K, const void *codes, int64_t pitch, const float *scales,
                                     void *X, void *stream);

/*
 * C = rne16(epi(alpha a_scales[m] w_scales[n] sum_k A[m][k] W[n][k])): M x N
 * binary16 row-major, 2-byte aligned, for A of M rows and W of N rows by K.
 * Sums are exact integers; a sum rounded to fp32 is multiplied by the fp32
 * product (alpha a_scales[m]) w_scales[n], then rounded once more to binary16.
 * (That product of scales has to be a finite fp32 number for a sum of 0, and
 * so for K = 0, to give +0.)  Limits: M <= GEMM_F16_MAX_DIM, N <=
 * GEMM_F16_MAX_N, pitches <= GEMM_F16_MAX_K.
 *   config : GEMM_F16_CONFIG_AUTO or an index below gemm_f16_i8_num_configs();
 *            all give the same bits.
 *   splits, workspace, workspace_bytes : as gemm_f16_split.  A split's partial
 *            sums are integers, so it gives the same bits too.
 */
gemm_f16_status_t gemm_f16_i8(int64_t M, int64_t N, int64_t K, const void *A, int64_t a_pitch, const float *a_scales,
                              const void *W, int64_t w_pitch, const float *w_scales, void *C, float alpha, int epilogue,
                              int config, int splits, void *workspace, int64_t workspace_bytes, void *stream);

/* How that call would run (no HIP call).  block_k is the k of one step,
 * k_tiles the steps of a split; vec_c is that of a 16-byte aligned C; flops
 * 2 M N K; min_bytes codes, scales and C once. */
gemm_f16_status_t gemm_f16_plan_i8(int64_t M, int64_t N, int64_t K, int config, int splits, gemm_f16_plan_t *plan);

int gemm_f16_i8_num_configs(void);
const char *gemm_f16_i8_config_name(int config);

/* ---- routed experts ------------------------------------------------------------
 * A token's logits choose top_k of `experts` experts.  The pair p = token
 * top_k + slot belongs to the expert ids[token][slot], or to none (an id that
 * is not in [0, experts)).  Limits: experts <= GEMM_F16_MAX_EXPERTS, top_k
 * <= GEMM_F16_MAX_TOP_K, groups <= GEMM_F16_MAX_EXPERT_GROUPS, tokens top_k <
 * 2^25.
 */
#define GEMM_F16_MAX_EXPERTS 1024
#define GEMM_F16_MAX_TOP_K 64
#define GEMM_F16_MAX_EXPERT_GROUPS 64
#define GEMM_F16_MAX_PAIRS (((int64_t)1 << 25) - 1)

#define GEMM_F16_SCORE_SOFTMAX 0
#define GEMM_F16_SCORE_SIGMOID 1

/*
 * Choose experts.  In 64 bits:
 *   score[e] = softmax over the token's experts, or sigmoid, of logit[e]
 *   key[e]   = score[e] + bias[e]
 * (bias NULL: the keys are the scores in the logits' order, that is, experts
 * whose scores round to the same number are compared by their logits).
 * An expert whose logit or bias is NaN or -inf is closed: its score is 0 and
 * it is never chosen.  A logit of +inf counts as the largest finite fp32.
 * With groups > 1 (it divides experts) the experts are `groups` blocks of
 * neighbours; the top_groups blocks with the largest sum of their two largest
 * score + bias (one: that one; bias NULL: scores) stay, those of equal sums
 * with the lowest indexes; blocks without an open expert never do.
 * ids[token] are the top_k experts with the largest keys among those left, the
 * largest first, equals in the order of their indexes; -1 from where there are
 * no more.
 *   weights[token][slot] = scale score[ids]               (renormalise 0)
 *                          scale score[ids] / sum of the chosen scores (1)
 * rounded to fp32; 0 for the id -1 and where the sum is 0.
 *   logits  : binary16 (half 1, 2-byte aligned) or fp32 (half 0), tokens rows
 *             of `experts`, stride >= experts elements apart.
 *   bias    : fp32, `experts` of them, or NULL.
 *   ids, weights : int32 and fp32, tokens x top_k.  scale: finite.
 */
gemm_f16_status_t gemm_f16_route(int64_t tokens, int experts, int top_k, const void *logits, int half, int64_t stride,
                                 int score, const float *bias, int groups, int top_groups, int renormalise, float scale,
                                 int32_t *ids, float *weights, void *stream);

/*
 * The pairs by expert: order holds the pairs p of expert 0, then of expert 1,
 * ... and at last those of none, each in ascending order; starts[e] (experts +
 * 1 of them) is the place of expert e's first pair, starts[experts] that of
 * the first pair of none.
 */
gemm_f16_status_t gemm_f16_expert_order(int64_t pairs, int experts, const int32_t *ids, int32_t *order, int32_t *starts,
                                        void *stream);

/*
 * The experts' products: for the pair p = order[i] of the expert e (starts[e]
 * <= i < starts[e + 1]),
 *   C[p] = rne16(epi(alpha a_scales[r] w_scales[e][n] sum_k A[r][k] W[e][n][k])),  r = p / pairs_per_row
 * as gemm_f16_i8 computes it, and zeros for the pairs of none.  A has
 * pairs / pairs_per_row rows: one for each token (pairs_per_row = top_k) or
 * one for each pair (1).  W: experts x N rows by K, w_scales experts x N.
 * Entries of order that are not in [0, pairs) are skipped; rows of C that
 * order does not name are left as they were.
 *   order, starts : as gemm_f16_expert_order gives them (starts not decreasing).
 *   config : GEMM_F16_CONFIG_AUTO or an index below gemm_f16_i8_num_configs().
 * Limits as gemm_f16_i8, and A of less than 2^31 bytes (for more, call it for
 * some of the tokens at a time, each time with their own order).
 */
gemm_f16_status_t gemm_f16_i8_experts(int64_t pairs, int64_t pairs_per_row, int experts, int64_t N, int64_t K,
                                      const void *A, int64_t a_pitch, const float *a_scales, const void *W,
                                      int64_t w_pitch, const float *w_scales, const int32_t *order,
                                      const int32_t *starts, void *C, float alpha, int epilogue, int config, void *stream);

/* How that call would run (no HIP call): tiles_m and grid are upper bounds,
 * vec_c is that of a 16-byte aligned C, flops 2 pairs N K; min_bytes all experts' codes and scales, A and C once. */
gemm_f16_status_t gemm_f16_plan_i8_experts(int64_t pairs, int64_t pairs_per_row, int experts, int64_t N, int64_t K,
                                           int config, gemm_f16_plan_t *plan);

/*
 * out[t] = rne16(sum over slots j of weights[t][j] Y[t][j]): Y tokens x top_k
 * x N binary16, weights fp32 tokens x top_k, out tokens x N binary16, all
 * contiguous.  Sums are fp32, in the order of the slots.  top_k = 0 writes zeros.
 */
gemm_f16_status_t gemm_f16_expert_sum(int64_t tokens, int64_t top_k, int64_t N, const void *Y, const float *weights,
                                      void *out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_F16_I8_H */
