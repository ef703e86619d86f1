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
 * them.  K = 0 writes +0.  Limits: M <= GEMM_F16_MAX_DIM, N and K as gemm_f16.
 *   config : GEMM_F16_CONFIG_AUTO or an index below gemm_f16_q4_num_configs().
 *            The tiles (plan: direct_lds 1) need A's rows 4-byte aligned (K
 *            even), the others nothing.  All of them use the weights s (q - z)
 *            exactly but the last one, q4_expanded: it runs gemm_f16_q4_expand
 *            into the workspace (2 N K bytes) and the dense product of
 *            gemm_f16_scaled, whose plan its own does not repeat, and so rounds
 *            each weight to binary16 (infinite from 65520 on) before the product.
 *            AUTO takes it from 2048 rows with groups of 32 and 64, where exact
 *            products take up to twice the time (but not for few outputs over
 *            K beyond 1024); never with splits 1.
 *   splits, workspace, workspace_bytes : as gemm_f16_split; the plan's
 *            workspace may also hold a copy of A with aligned rows (K odd).
 *            splits 1 with config AUTO never needs a workspace, and uses every
 *            weight exactly.
 */
gemm_f16_status_t gemm_f16_q4(int64_t M, int64_t N, int64_t K, int group, const void *A, const void *codes,
                              const void *words, void *C, float alpha, int epilogue, int config, int splits,
                              void *workspace, int64_t workspace_bytes, void *stream);

/* How that call would run (no HIP call; A only for its alignment, NULL for an
 * aligned one).  block_k is the k of one step, k_tiles the steps of a split;
 * flops 2 M N K; min_bytes the codes and words, A and C once. */
gemm_f16_status_t gemm_f16_plan_q4(int64_t M, int64_t N, int64_t K, int group, const void *A, int config, int splits,
                                   gemm_f16_plan_t *plan);

int gemm_f16_q4_num_configs(void);
const char *gemm_f16_q4_config_name(int config);

/* ---- key/value cache ---------------------------------------------------------
 * Keys and values of `heads` heads of `head_dim` (64, 128 or 256) in `pages`
 * pages of `page_size` tokens (a multiple of 8), rounded per token and head
 * in groups of `group` neighbours of the head dimension (group <= head_dim).
 * Codes and words, uint32, contiguous, 16-byte aligned:
 *   k_codes [pages][heads][page_size][head_dim / 8]; in every block of
 *           b = min(head_dim, 128) the dword of d = 32 j + 8 g + 0..7 is at
 *           g (b / 32) + j
 *   v_codes [pages][heads][page_size / 8][16][head_dim / 16]: [d % 16][d / 16]
 *           holds 8 successive tokens of one d, token i of the eight as value i
 *   k_words, v_words [pages][heads][head_dim / group][page_size]
 * A sequence's token t is in slot t % page_size of page table[t / page_size]
 * of its row of the page table.
 */
typedef struct gemm_f16_q4_cache {
    void *k_codes, *k_words, *v_codes, *v_words;
    int64_t pages;
    int32_t heads, page_size, head_dim, group;
} gemm_f16_q4_cache_t;

/* Limits (beyond them, where a launch would have 2^32 work items or more, and
 * where a buffer would have more than 2^56 bytes:
 * GEMM_F16_ERROR_UNSUPPORTED_SIZE). */
#define GEMM_F16_Q4_MAX_HEADS 4096
#define GEMM_F16_Q4_MAX_BATCH ((int64_t)1 << 20)
#define GEMM_F16_Q4_MAX_PAGE ((int64_t)1 << 16)
#define GEMM_F16_Q4_MAX_LENGTH ((int64_t)1 << 30)   /* max_pages * page_size */
#define GEMM_F16_Q4_MAX_TOKENS ((int64_t)1 << 26)   /* of one append or read */
#define GEMM_F16_Q4_MAX_PAGES ((int64_t)1 << 30)

/*
 * Append new tokens' keys and values to the cache.
 *   K, V    : tokens x heads x head_dim binary16; a token's heads are
 *             contiguous, tokens k_stride / v_stride elements apart (slices
 *             of a fused projection's output need no copy).
 *   table   : int32 batch x max_pages.
 *   lengths : int32 batch, tokens already in the cache.
 *   starts  : int32 batch + 1: sequence i's new tokens are rows starts[i] up
 *             to starts[i + 1] (not decreasing).  NULL: one token for each
 *             sequence (tokens == batch).
 *   cos, sin: fp32 positions x rotary_dim / 2, or NULL (no rotation):
 *             rotation of the first rotary_dim (a multiple of 16) elements of
 *             keys (and Q) by the angle of the token's position, of the pairs
 *             (i, i + rotary_dim / 2), or (2 i, 2 i + 1) with interleaved 1:
 *             (a, b) -> (a cos - b sin, b cos + a sin), in fp32, rounded only
 *             to codes (Q: to binary16).
 *   Q, Q_out: queries of the same tokens, tokens x q_heads x head_dim
 *             (q_stride elements apart), rotated into Q_out (contiguous);
 *             both NULL: none.  Q_out may be Q when Q is contiguous.
 * New token j of sequence i goes to position lengths[i] + j.  A token is not
 * written, and its row of Q_out is zeroed, when its position is negative,
 * past max_pages * page_size or (with cos) not below positions, or its page is
 * not in [0, pages).  Rows of no sequence are left as they were, in the
 * cache and in Q_out.  A granule, 8 slots of a page from a multiple of 8 on, is
 * appended to from one place: not by two sequences, nor by one whose table
 * names the page twice (what the granule then holds of the new tokens is
 * undefined; other granules of the page are not touched by it).
 */
gemm_f16_status_t gemm_f16_q4_cache_append(const gemm_f16_q4_cache_t *cache, int64_t batch, int64_t tokens,
                                           int64_t max_pages, const void *K, int64_t k_stride, const void *V,
                                           int64_t v_stride, const int32_t *table, const int32_t *lengths,
                                           const int32_t *starts, const void *Q, int64_t q_stride, void *Q_out,
                                           int q_heads, const float *cos, const float *sin, int64_t positions,
                                           int rotary_dim, int interleaved, void *stream);

/*
 * What the cache holds of each sequence: row starts[i] + j of K and V
 * (tokens x heads x head_dim binary16, contiguous, 16-byte aligned) becomes
 * position first[i] + j (first NULL: from 0), each value rounded once; zeros
 * for a position or page out of range.  Rows of no sequence are left.
 */
gemm_f16_status_t gemm_f16_q4_cache_read(const gemm_f16_q4_cache_t *cache, int64_t batch, int64_t tokens,
                                         int64_t max_pages, const int32_t *table, const int32_t *first,
                                         const int32_t *starts, void *K, void *V, void *stream);

/*
 * Attention of one query token of each sequence over its cached keys and
 * values, the score block scaled as gemm_f16_scaled's:
 *   out[i][h] = sum_t softmax_t(scale * q[i][h] . k[t]) v[t],  t < lengths[i]
 * with query head h reading cache head h / (q_heads / heads).
 *   Q, out  : batch x q_heads x head_dim binary16; Q's sequences q_stride
 *             elements apart, out contiguous (16-byte aligned both, q_stride
 *             a multiple of 8); out overlaps nothing else.
 *   lengths : int32 batch; a length below 1 gives a row of zeros, one beyond
 *             max_pages * page_size counts as that.  Tokens whose page is not
 *             in [0, pages) are left out, as by a mask.
 *   splits  : parts the sequences are divided into, computed by separate
 *             workgroups and joined in order by a second kernel:
 *             GEMM_F16_SPLITS_AUTO or 1 .. GEMM_F16_Q4_MAX_SPLITS.
 *   scale   : finite.
 *   max_length : what no length exceeds, for the choice of splits only (0:
 *             max_pages * page_size); any value gives right results.
 *   workspace : caller-owned, 16-byte aligned, of at least the plan's
 *             workspace_bytes, as gemm_f16_split's; NULL when the plan has 1
 *             split.
 * Scores, softmax and sums are fp32; codes enter the matrix cores exactly and
 * probabilities times scales in two binary16 parts, under a power of two for
 * each group of d whose scales lie far from the others'; one rounding at the end.
 */
#define GEMM_F16_Q4_MAX_SPLITS 256
gemm_f16_status_t gemm_f16_q4_attention(const gemm_f16_q4_cache_t *cache, int64_t batch, int q_heads,
                                        int64_t max_pages, const void *Q, int64_t q_stride, const int32_t *table,
                                        const int32_t *lengths, float scale, void *out, int splits,
                                        int64_t max_length, void *workspace, int64_t workspace_bytes, void *stream);

/* How that call would run, without any HIP call: splits, workspace_bytes,
 * grid (workgroups of the first kernel), threads, lds_bytes, block_m (query
 * heads of a workgroup), block_n (tokens of a wave's step); flops and
 * min_bytes of max_length tokens in every sequence. */
gemm_f16_status_t gemm_f16_plan_q4_attention(int64_t batch, int q_heads, int heads, int head_dim, int group,
                                             int64_t max_length, int splits, gemm_f16_plan_t *plan);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_F16_Q4_H */
