/*
 * gemm_f16_q4.h -- C ABI of the products with 4-bit operands of the FP16 GEMM
 * library for AMD Instinct MI355X (gfx950): weights and key/value caches held
 * as 4-bit codes with a scale and a zero point for every group.
 *
 * The pages whose tile GEMM the library implements name these operators among
 * the ones built on the same tiles: dequantised products and attention
 * ("5分钟上手TileLang：GPU内核开发指南", section "进阶方向：从 GEMM 到真实模型算子";
 * "TileLang：比 Triton 低一层的 tile 语言", section "FlashAttention：在线
 * softmax 写成 tile 代码"), without a storage format.  The format is the
 * library's own.
 *
 * Format.  A group is `group` (32, 64 or 128) neighbours along the
 * contraction (weights) or the head dimension (cache).  It has one 32-bit
 * word: a binary16 scale s in the low half, an integer zero point z (0..15)
 * in the high half.  A code q (0..15) stands for s (q - z).  Eight
 * consecutive values share a dword: value i of the eight is the nibble at
 * bits 4 p(i) .. 4 p(i) + 3 with p = 0, 4, 1, 5, 2, 6, 3, 7.  (With that
 * order one mask and one OR give two neighbouring codes as binary16.)
 *
 * Rounding to codes: x is decoded exactly; lo = min(0, smallest x of the
 * group), hi = max(0, largest), in fp32.
 *   asymmetric: s = rne16(min((hi - lo) / 15, 65504)), z = clamp(rint(-lo / s), 0, 15)
 *   symmetric:  s = rne16(min(max |x| / 7, 65504)),    z = 8
 *   q = clamp(rint(x / s) + z, 0, 15), and q = z (asymmetric: 0) where s = 0.
 * NaN counts as 0, infinities saturate.
 *
 * Ownership, streams, errors: as in gemm_f16.h.  Buffers belong to the
 * caller, nothing is allocated, nothing synchronises, every entry point may
 * be captured into a HIP graph, and results are bitwise reproducible.
 * Arguments are validated before any HIP call; on error nothing is launched.
 */
#ifndef GEMM_F16_Q4_H
#define GEMM_F16_Q4_H

#include "gemm_f16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- weights ---------------------------------------------------------------
 * W (N x K binary16 row-major: the B of gemm_f16_trans given N x K) is held
 * in tiles of 16 rows by 128 k, the last row and column of tiles padded with
 * zeros.  With NB = ceil(N / 16) and KB = ceil(K / 128):
 *   codes : uint32 [NB][KB][4 g][16 n][4 j]; the dword holds row n of the
 *           tile, k = 32 j + 8 g + 0..7 of the tile.  A tile is 1 KiB, in the
 *           order in which the 64 lanes of a wave feed the matrix cores.
 *   words : uint32 [NB][KB][16 n][128 / group], the groups of row n in order.
 */

/* Bytes of the two buffers, or -1 for a negative or too large dimension or
 * an unknown group (words). */
int64_t gemm_f16_q4_codes_bytes(int64_t N, int64_t K);
int64_t gemm_f16_q4_words_bytes(int64_t N, int64_t K, int group);

/* Round W to codes and words (both written whole, padding included).  W needs
 * 2-byte alignment, codes and words 16-byte; none may overlap. */
gemm_f16_status_t gemm_f16_q4_compress(int64_t N, int64_t K, int group, int symmetric, const void *W,
                                       void *codes, void *words, void *stream);

/* W = rne16(s (q - z)), N x K row-major. */
gemm_f16_status_t gemm_f16_q4_expand(int64_t N, int64_t K, int group, const void *codes, const void *words,
                                     void *W, void *stream);

/*
 * C = rne16(epi(alpha * A . W^T)) for A (M x K), C (M x N) binary16
 * row-major and W held as (codes, words).  Meant for few rows (M = 1 is one
 * token through a layer: each code is read once) and right for any M >= 0.
 * A and C need 2-byte alignment, codes and words 16-byte; C overlaps none of
 * them.  K = 0 writes +0.  config: GEMM_F16_CONFIG_AUTO or an index below
 * gemm_f16_q4_num_configs(); every configuration runs every shape.
 * Limits: M <= GEMM_F16_MAX_DIM, N and K as gemm_f16.
 */
gemm_f16_status_t gemm_f16_q4(int64_t M, int64_t N, int64_t K, int group, const void *A, const void *codes,
                              const void *words, void *C, float alpha, int epilogue, int config, void *stream);

/* How that call would run (no HIP call).  block_k is the k of one step of a
 * wave, k_tiles the steps of all of K; flops 2 M N K; min_bytes the codes and
 * words, A and C once. */
gemm_f16_status_t gemm_f16_plan_q4(int64_t M, int64_t N, int64_t K, int group, int config,
                                   gemm_f16_plan_t *plan);

int gemm_f16_q4_num_configs(void);
const char *gemm_f16_q4_config_name(int config);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_F16_Q4_H */
