// gemm_f16_q4_api.cpp -- the C ABI of the products with 4-bit operands:
// argument validation, choice of kernel and launch.  Validation and planning
// make no HIP call.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <cmath>

#include "gemm_f16_internal.h"
#include "gemm_f16_q4.h"
#include "gemm_f16_q4_format.h"

namespace gemm_f16_impl {

const Q4Config kQ4Configs[kNumQ4Configs] = {
    {"q4_16x16", 1, 1, 8, 0},
    {"q4_16x32", 1, 2, 8, 0},
    {"q4_16x64", 1, 4, 8, 0},
    {"q4_32x64", 2, 4, 8, 0},
    {"q4_32x128", 2, 8, 8, 0},
    {"q4_64x128_s4", 4, 8, 8, 4},
    {"q4_128x256_s3", 8, 16, 8, 3},
    {"q4_expanded", 0, 0, 0, 0},
};

int64_t q4_lds_bytes(const Q4Config &c, int group)
{
    if (c.stages == 0)   // (no waves, no LDS: the expanded product's is its own)
        return (int64_t)c.waves * c.m_blocks * q4_sum_chunk(c.m_blocks, c.n_blocks) * 1024;
    const int64_t word_loads = (c.n_blocks * (128 / group) / 4 + c.waves - 1) / c.waves;
    return std::max<int64_t>(c.stages * (c.m_blocks * 4096 + c.n_blocks * 1024 + c.waves * word_loads * 256),
                             16 * c.m_blocks * (16 * c.n_blocks + 8) * 2);
}

namespace {

bool known_group(int group) { return group == 32 || group == 64 || group == 128; }

// Work items of a launch's grid are counted in 32 bits.
bool launchable(int64_t workgroups, int64_t threads) { return workgroups <= 0xffffffff / threads; }

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

// Whether the tile kernels' direct loads can read A's rows.
bool rows_4_aligned(const void *A, int64_t K) { return (uintptr_t)A % 4 == 0 && K % 2 == 0; }

// Rows of A that are not 4-byte aligned (an odd K or pointer) are first copied
// to aligned rows in the workspace, where one is allowed and there are enough
// of them: every kernel but the one that loads single elements becomes possible.
// us at (M, N x K) without and with the copy: (48, 8192 x 8193) 57, 24; (300, 4096 x
// 4097) 68, 31; (1000, 8192 x 8193) 490, 154; (2100, 8192 x 8193) 1040, 386; (16, 4096 x
// 4097) 14.9, 7.9; (8, 8192 x 8193) 20.9, 14.6; but (16, 20000 x 1001) 9.3, 9.6, (8, 20000 x
// 1001) 8.4, 9.1 and (1, 8192 x 8193) 11.6, 14.0.
bool packs(int64_t M, int64_t N, int64_t K, bool aligned, int config, int splits)
{
    return !aligned && config == GEMM_F16_CONFIG_AUTO && splits == GEMM_F16_SPLITS_AUTO &&
           (M >= 16 || (M >= 8 && K >= 4096)) && N > 0 && K > 0;
}
int64_t packed_k(int64_t K) { return (K + 7) / 8 * 8; }   // within the last group: the codes' order is the same
int64_t packed_bytes(int64_t M, int64_t K) { return (2 * M * packed_k(K) + 255) / 256 * 256; }

gemm_f16_status_t make_plan(int64_t M, int64_t N, int64_t K, int group, bool aligned, int config, int splits,
                            gemm_f16_plan_t *p)
{
    if (packs(M, N, K, aligned, config, splits)) {
        const gemm_f16_status_t st = make_plan(M, N, packed_k(K), group, true, config, splits, p);
        p->workspace_bytes += packed_bytes(M, K);
        p->flops = 2.0 * (double)M * (double)N * (double)K;
        return st;
    }
    if ((config != GEMM_F16_CONFIG_AUTO && (config < 0 || config >= kNumQ4Configs)) || splits < 0 ||
        splits > GEMM_F16_MAX_SPLITS)
        return GEMM_F16_ERROR_INVALID_VALUE;
    // Few rows.  Wider workgroups read A and W less often, but leave CUs idle
    // when they are few: the widest one that makes 150 workgroups.  us at (M, N x
    // K) for 16x16 / 16x32 / 16x64 / 32x64 / 32x128, * the choice: (1, 4096 x 4096) *4.4 /
    // 5.6 / 7.5; (1, 8192 x 8192) 11.1 / *10.6 / 14.6; (1, 28672 x 8192) 35.4 / 28.3 / *26.2;
    // (16, 28672 x 8192) 57.4 / 41.1 / *33.1; (16, 5000 x 4100) 9.1 / *7.5 / 8.7; (48, 5000 x 4100)
    // 14.8 / 11.5 / 10.2 / *11.9 / 14.8; (64, 4096 x 4096) - / - / *9.0 / 10.7 / 13.3.
    // With 64 blocks of K or more, splitting K beats narrower workgroups:
    // (24, 2048 x 16384) 18.1 / 13.5 / 12.0 / *11.9 / 13.9; (24, 8192 x 8192) 29.2 / 19.1 /
    // 15.8 / *14.4 / 16.7; and from 33 rows the 64x128 tile does (us, best of the
    // others): (48, 8192 x 8192) 20, 22; (64, 28672 x 8192) 53, 65; (128, 4096 x 14336)
    // 29, 31; but (32, 8192 x 8192) 18.2, 16.9 and (64, 5000 x 4100) 13.5, 12.8.  Between 4096 and
    // 8192 of K the border moves with N, within 15 %: (64, 8192 x 7168) 18.8, 20.6; (64, 4096 x
    // 7168) 14.7, 13.7; (64, 2048 x 8064) 13.9, 12.1; (64, 8192 x 5120) 16.4, 15.6.
    // It also does where the widest workgroup would come in more than one round, as
    // it starts and ends faster: (64, 28672 x 4096) 28, 39; (128, 14336 x 512) 6.8, 11.8;
    // (300, 5000 x 1024) 9.7, 15.3; (300, 4096 x 4096) 25, 33; but (128, 8192 x 4096) 21.2, 18.8.
    // The 128x256 tile takes over where it makes 64 workgroups for more than
    // 64 rows (its time, the 64x128 tile's, with groups of 64): (100, 28672 x 8192) 80, 100;
    // (200, 8192 x 8192) 47, 49; (1500, 5000 x 4100) 72, 111; but (200, 4096 x 4096) 28, 18,
    // (128, 8192 x 8192) 34, 30 and (64, 28672 x 8192) 74, 53; and not while the 64x128
    // tile's workgroups are one round over at most 32 blocks of K, or two over 16:
    // (512, 4096 x 4096) 35, 26; (256, 8192 x 1024) 20, 9; (1024, 4096 x 2048) 35, 28; but
    // (1024, 4096 x 4096) 50, 51 and (512, 14336 x 1024) 22, 31.
    // Both tiles use weights exactly.  From 2048 rows, W expanded to binary16 and
    // the dense product take less time, but each weight is rounded.  That is only
    // accepted where it saves most: exact products with groups of 128 take a third
    // longer at most, so they stay exact; with groups of 64 they take up to half
    // as long again, with 32 twice as long.  (us, the tile's with groups of 128, 64,
    // 32, and this) (2048, 8192 x 8192) 244, 279, 372, 201; (8192, 8192 x 8192) 952, 1094,
    // 1480, 720; (8192, 2048 x 2048) 71, 86, 105, 57; (2048, 5000 x 4100) 128, 131, 185, 126; but
    // fewer rows, (1024, 8192 x 8192) 125, 141, 187, 132, gain less, and (1536, 8192 x 28672) 739, 919,
    // 1279, 950.  Not where the caller allows no workspace (1 split).
    // The dense product does not split K: it needs 2^21 outputs (N in whole tiles of
    // 64) to fill the card, over K of 1024 or less 2^23 to be worth the rounding.  (The
    // tile's time, this one's, groups of 64) (2048, 64 x 8192) 14, 32; (2048, 256 x 16384) 32,
    // 60; (2048, 512 x 8192) 32, 37; (2048, 2048 x 1024) 18, 23; but (2048, 2048 x 8192) 88, 64;
    // (8192, 256 x 8192) 54, 49; (30000, 128 x 8192) 120, 106 and (8192, 2048 x 1024) 45, 35.
    // Fewer outputs over such a K take either way 5 to 10 us, within 1.5 of each other.
    const int64_t n_blocks = (N + 15) / 16, blocks = (K + 127) / 128;
    const int large = kQ4Expanded - 1, most_m = M > 16 ? 2 : 1;
    const int64_t outputs = M * ((N + 63) / 64 * 64);
    const bool expands = M >= 2048 && group < 128 && K > 0 &&
                         (K > 1024 ? outputs >= 1 << 21 : outputs < 1 << 21 || outputs >= 1 << 23);
    const auto count = [&](int i) {
        const int64_t m = 16 * kQ4Configs[i].m_blocks, n = kQ4Configs[i].n_blocks;
        return (M + m - 1) / m * ((n_blocks + n - 1) / n);
    };
    int c = config;
    if (c == GEMM_F16_CONFIG_AUTO) {
        if (expands && N > 0 && splits == GEMM_F16_SPLITS_AUTO) {
            c = kQ4Expanded;
        } else if (aligned && M > 64 && count(large) >= 64 && count(large - 1) > (blocks <= 16 ? 512 : blocks <= 32 ? 256 : 0)) {
            c = large;
        } else if (aligned && M > 32 && (blocks >= 64 || count(large - 2) > 256)) {
            c = large - 1;
        } else {
            for (c = large - 2; c > 0; --c)
                if (kQ4Configs[c].m_blocks <= most_m && count(c) >= 150)
                    break;
            if (M > 8 && blocks >= 64)
                c = std::max(c, M > 16 ? 3 : 2);
        }
    }
    const Q4Config &d = kQ4Configs[c];
    if ((d.stages > 0 && !aligned) || (c == kQ4Expanded && splits > 1))
        return GEMM_F16_ERROR_INVALID_VALUE;
    memset(p, 0, sizeof(*p));
    p->config = c;
    p->flops = 2.0 * (double)M * (double)N * (double)K;
    p->min_bytes = 0.5 * (double)N * (double)K + 4.0 * (double)N * (double)((K + group - 1) / group) +
                   2.0 * (double)M * ((double)N + (double)K);
    p->trans_b = 1;
    if (c == kQ4Expanded) {   // the rest is the dense product's own plan
        p->splits = 1;
        p->k_split = K;
        p->workspace_bytes = M > 0 ? 2 * N * K : 0;
        return GEMM_F16_SUCCESS;
    }
    p->block_m = 16 * d.m_blocks;
    p->block_n = 16 * d.n_blocks;
    p->block_k = 128;
    p->stages = d.stages > 0 ? d.stages : 1;
    p->threads = 64 * d.waves;
    p->direct_lds = d.stages > 0;
    p->vec_a = d.stages > 0 ? 2 : 1;
    p->vec_b = 32;
    p->vec_c = 8;
    p->tiles_m = (M + p->block_m - 1) / p->block_m;
    p->tiles_n = (N + p->block_n - 1) / p->block_n;
    const int64_t tiles = p->tiles_m * p->tiles_n;
    if (splits == GEMM_F16_SPLITS_AUTO) {
        splits = 1;
        if (M > 8 && tiles > 0 && tiles < (d.stages > 0 ? 256 : 150))   // a part keeps 8 blocks, two for each wave of the kernel for few rows
            splits = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(256 / tiles, blocks / (d.stages > 0 ? 8 : 16)),
                                                                 GEMM_F16_MAX_SPLITS));
        // one row or few, where it saves more than the second launch costs a caller
        // that does not capture its calls, 3 us.  us whole and split: (1, 1024 x 28672)
        // 16.0, 8.2; (4, 1024 x 16384) 11.6, 7.5; (1, 256 x 16384) 10.1, 6.1; but (1, 512 x
        // 8192) 6.2, 5.4, (8, 2048 x 8192) 8.1, 7.4, (1, 512 x 4096) 3.8, 4.9, (4, 4096 x 8192)
        // 7.3, 9.2, and in 8 parts (1, 1024 x 28672) 8.5 and (4, 1024 x 16384) 8.9.
        else if (M <= 8 && d.stages == 0 && blocks >= 128 && tiles > 0 && tiles <= 128)
            splits = (int)std::min<int64_t>(std::min<int64_t>(256 / tiles, blocks / 16), 4);
    }
    const int64_t per = blocks > 0 ? (blocks + splits - 1) / splits : 0;
    p->splits = per > 0 ? (int)((blocks + per - 1) / per) : 1;   // none empty
    p->grid = tiles * p->splits;
    p->k_tiles = per;
    p->k_split = p->splits > 1 ? per * 128 : K;
    p->lds_bytes = q4_lds_bytes(d, group);
    p->workspace_bytes = p->splits > 1 ? (int64_t)p->splits * M * N * 4 : 0;
    return d.stages > 0 && !launchable(p->grid, p->threads) ? GEMM_F16_ERROR_UNSUPPORTED_SIZE : GEMM_F16_SUCCESS;
}

// More bytes than an address space has: sizes are refused before their product
// in 64 bits, or an address plus it, could overflow.
constexpr int64_t kMostBytes = (int64_t)1 << 56;

// The cache's description and the page table's shape.
gemm_f16_status_t validate_cache(const gemm_f16_q4_cache_t *c, int64_t batch, int64_t max_pages)
{
    if (!c || c->pages < 0 || c->heads < 1 || batch < 0 || max_pages < 0 || !known_group(c->group) ||
        (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) || c->group > c->head_dim || c->page_size < 8 ||
        c->page_size % 8 != 0)
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (c->heads > GEMM_F16_Q4_MAX_HEADS || batch > GEMM_F16_Q4_MAX_BATCH || c->page_size > GEMM_F16_Q4_MAX_PAGE ||
        c->pages > GEMM_F16_Q4_MAX_PAGES || max_pages > GEMM_F16_Q4_MAX_LENGTH / c->page_size)
        return GEMM_F16_ERROR_UNSUPPORTED_SIZE;
    // (a page's codes have at most 2^35 bytes, its words a quarter of that)
    if (c->pages > kMostBytes / ((int64_t)c->heads * c->page_size * (c->head_dim / 2)))
        return GEMM_F16_ERROR_UNSUPPORTED_SIZE;
    if (c->pages > 0 && (!c->k_codes || !c->k_words || !c->v_codes || !c->v_words))
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (((uintptr_t)c->k_codes | (uintptr_t)c->k_words | (uintptr_t)c->v_codes | (uintptr_t)c->v_words) % 16)
        return GEMM_F16_ERROR_MISALIGNED;
    return GEMM_F16_SUCCESS;
}

// Bytes of k_codes (and v_codes), and of k_words (and v_words), at most
// kMostBytes once the cache is validated.
int64_t cache_codes_bytes(const gemm_f16_q4_cache_t *c)
{
    return c->pages * c->heads * c->page_size * (c->head_dim / 2);
}
int64_t cache_words_bytes(const gemm_f16_q4_cache_t *c)
{
    return c->pages * c->heads * c->page_size * (c->head_dim / c->group) * 4;
}

// Whether a range shares a byte with any of the cache's buffers.
bool overlaps_cache(const void *p, int64_t bytes, const gemm_f16_q4_cache_t *c)
{
    const int64_t cb = cache_codes_bytes(c), wb = cache_words_bytes(c);
    return overlaps(p, bytes, c->k_codes, cb) || overlaps(p, bytes, c->v_codes, cb) ||
           overlaps(p, bytes, c->k_words, wb) || overlaps(p, bytes, c->v_words, wb);
}

bool buffers_apart(const gemm_f16_q4_cache_t *c)
{
    const int64_t cb = cache_codes_bytes(c), wb = cache_words_bytes(c);
    return !overlaps(c->k_codes, cb, c->v_codes, cb) && !overlaps(c->k_codes, cb, c->k_words, wb) &&
           !overlaps(c->k_codes, cb, c->v_words, wb) && !overlaps(c->v_codes, cb, c->k_words, wb) &&
           !overlaps(c->v_codes, cb, c->v_words, wb) && !overlaps(c->k_words, wb, c->v_words, wb);
}

Q4Pages pages_of(const gemm_f16_q4_cache_t *c, const int32_t *table, int64_t batch, int64_t max_pages)
{
    Q4Pages p;
    p.k_codes = (uint32_t *)c->k_codes;
    p.k_words = (uint32_t *)c->k_words;
    p.v_codes = (uint32_t *)c->v_codes;
    p.v_words = (uint32_t *)c->v_words;
    p.pages = c->pages;
    p.heads = c->heads;
    p.page_size = c->page_size;
    p.head_dim = c->head_dim;
    p.group = c->group;
    p.table = table;
    p.batch = (int)batch;
    p.max_pages = (int)max_pages;
    // t / d = floor(t m / 2^(31 + n)) with 2^(n-1) < d <= 2^n and m = floor(2^(31 + n) / d) + 1: m d exceeds
    // 2^(31 + n) by at most d, so the quotient is off by at most t / 2^(31 + n) < 1 / d for t < 2^31
    int n = 3;
    while ((1 << n) < c->page_size)
        ++n;
    p.page_magic = (uint32_t)(((uint64_t)1 << (31 + n)) / (uint64_t)c->page_size + 1);
    p.page_shift = n - 1;
    return p;
}

// Rows of `heads` heads at a pitch of `stride` elements: long enough, within an
// address space, and whether 16-byte loads are aligned.
bool rows_fit(int64_t stride, int64_t heads, int head_dim) { return stride >= heads * head_dim; }
bool rows_reach(int64_t rows, int64_t stride) { return rows <= 0 || stride <= kMostBytes / 2 / rows; }
bool rows_aligned(const void *p, int64_t stride) { return (uintptr_t)p % 16 == 0 && stride % 8 == 0; }
int64_t rows_bytes(int64_t rows, int64_t stride, int64_t width) { return rows > 0 ? 2 * ((rows - 1) * stride + width) : 0; }

// Blocks of 32 tokens that a wave takes at once.  The 16 columns of its products
// are query heads; where 4 or 8 heads share a cache head, the softmax of 4 or 2
// blocks goes through the columns together (32 x 4096 tokens x 8 heads, 4 query
// heads each: 26.2 us with 4 blocks, 28.1 with 2, 28.6 with 1), while that leaves
// steps for a wave on every SIMD (8 heads of one sequence of 2000: 7.5 us with 1
// block, 8.0 with 2, 9.7 with 4).  head_dim 256 has registers for 2.
//
// Parts of the sequences: none where every CU has two workgroups without
// (64 x 1000 tokens x 8 heads: 15.9 us whole, 21.6 in two parts); else as many
// as make two for each CU, or four where sequences may differ in length and
// the next workgroup evens that out (32 x 4096 x 8 heads: 26.2 us in four parts,
// 28.3 in two, 29.1 whole; one sequence of 131000: 34.2 us in 64 parts, 35.8 in 128),
// for head_dim 256 what its registers admit at once (4 x 8000 x 4 heads: 16.2 us
// in 16 parts, 19.4 in 32, 21.6 in 8), down to a block of tokens for each wave of a
// part (one sequence of 2000: 7.5 us in 16 parts, 8.2 in 8).  The second kernel
// costs 2 us at least, so short sequences stay whole (16 x 4 heads of 64 / 128 /
// 256, whole or in parts: 380 tokens 5.0, 6.4, 10.0 or 6.6, 7.2, 8.7 us; 200
// tokens 4.4, 5.4, 7.9 or 6.5, 7.2, 8.5; 640 tokens 6.4, 8.5, 13.8 or 7.2, 8.4, 10.0).
// (Since the exponents of P' follow their groups, times are 1 to 4 % above these.)
// A table wider than the sequences costs up to a quarter where max_length does not
// say so: 8 x 1000 tokens 8.0 us, 10.0 with room for 32768; one of 2000 7.7, 9.3.
gemm_f16_status_t plan_attention(int64_t batch, int q_heads, int heads, int head_dim, int group, int64_t max_length,
                                 int splits, gemm_f16_plan_t *p)
{
    if (batch < 0 || q_heads < 1 || heads < 1 || q_heads % heads != 0 || max_length < 0 || splits < 0 ||
        splits > GEMM_F16_Q4_MAX_SPLITS || !known_group(group) || group > head_dim ||
        (head_dim != 64 && head_dim != 128 && head_dim != 256))
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (batch > GEMM_F16_Q4_MAX_BATCH || q_heads > GEMM_F16_Q4_MAX_HEADS || max_length > GEMM_F16_Q4_MAX_LENGTH)
        return GEMM_F16_ERROR_UNSUPPORTED_SIZE;
    const int64_t ratio = q_heads / heads, tiles = (ratio + 15) / 16, units = batch * heads * tiles;
    const int64_t blocks = (max_length + kQ4AttentionTokens - 1) / kQ4AttentionTokens;
    int sub = ratio <= 4 && head_dim < 256 ? 4 : ratio <= 8 ? 2 : 1;
    while (sub > 1 && units * blocks / sub < 4 * 256)
        sub /= 2;
    if (splits == GEMM_F16_SPLITS_AUTO) {
        const int64_t here = head_dim == 256 && group < 128 ? 256 : 2 * 256;
        const int64_t fill = units <= 0 || units >= here ? 1 : (batch > 1 && head_dim < 256 ? 2 * here : here) / units;
        const int64_t most = (blocks + kQ4AttentionWaves - 1) / kQ4AttentionWaves;
        splits = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(fill, most), GEMM_F16_Q4_MAX_SPLITS));
        if (blocks <= std::min(20, 1920 / head_dim))
            splits = 1;
    }
    memset(p, 0, sizeof(*p));
    p->block_m = 16;
    p->block_n = sub * kQ4AttentionTokens;
    p->block_k = head_dim;
    p->stages = 1;
    p->threads = 64 * kQ4AttentionWaves;
    p->vec_a = p->vec_c = 8;
    p->vec_b = 32;
    p->tiles_m = batch * heads * tiles;
    p->tiles_n = splits;
    p->grid = units * splits;
    p->lds_bytes = q4_attention_lds_bytes(head_dim);
    p->flops = 4.0 * (double)batch * (double)max_length * (double)q_heads * (double)head_dim;
    p->min_bytes = (double)batch * ((double)max_length * heads * (head_dim + 8.0 * head_dim / group) + 4.0 * q_heads * head_dim);
    p->splits = splits;
    p->workspace_bytes = splits > 1 ? batch * q_heads * splits * (head_dim + 2) * 4 : 0;
    return launchable(p->grid, p->threads) && launchable(batch * q_heads, 256) ? GEMM_F16_SUCCESS : GEMM_F16_ERROR_UNSUPPORTED_SIZE;
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
                                        symmetric != 0, (hipStream_t)stream));
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
                                      (hipStream_t)stream));
}

gemm_f16_status_t gemm_f16_q4(int64_t M, int64_t N, int64_t K, int group, const void *A, const void *codes,
                              const void *words, void *C, float alpha, int epilogue, int config, int splits,
                              void *workspace, int64_t workspace_bytes, void *stream)
{
    gemm_f16_status_t st = validate_weights(N, K, group, codes, words);
    if (st != GEMM_F16_SUCCESS)
        return st;
    if (M < 0 || (epilogue != GEMM_F16_EPILOGUE_NONE && epilogue != GEMM_F16_EPILOGUE_RELU) || workspace_bytes < 0 ||
        (!workspace && workspace_bytes != 0))
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
    st = make_plan(M, N, K, group, rows_4_aligned(A, K), config, splits, &plan);
    if (st != GEMM_F16_SUCCESS)
        return st;
    if (M == 0 || N == 0)
        return GEMM_F16_SUCCESS;
    if (plan.workspace_bytes > 0) {
        if (!workspace)
            return GEMM_F16_ERROR_WORKSPACE;
        if ((uintptr_t)workspace % 16)
            return GEMM_F16_ERROR_MISALIGNED;
        if (workspace_bytes < plan.workspace_bytes)
            return GEMM_F16_ERROR_WORKSPACE;
        const int64_t wb = plan.workspace_bytes;
        if (overlaps(workspace, wb, A, 2 * M * K) || overlaps(workspace, wb, C, 2 * M * N) ||
            overlaps(workspace, wb, codes, gemm_f16_q4_codes_bytes(N, K)) ||
            overlaps(workspace, wb, words, gemm_f16_q4_words_bytes(N, K, group)))
            return GEMM_F16_ERROR_INVALID_VALUE;
    }
    int dev = -1;
    st = check_device(&dev);
    if (st != GEMM_F16_SUCCESS)
        return st;
    if (packs(M, N, K, rows_4_aligned(A, K), config, splits)) {
        if (launch_q4_pack((const _Float16 *)A, (_Float16 *)workspace, M, K, packed_k(K), (hipStream_t)stream) != hipSuccess)
            return GEMM_F16_ERROR_LAUNCH_FAILED;
        const int64_t used = packed_bytes(M, K), rest = plan.workspace_bytes - used;
        return gemm_f16_q4(M, N, packed_k(K), group, workspace, codes, words, C, alpha, epilogue, config, splits,
                           rest > 0 ? (char *)workspace + used : nullptr, rest, stream);
    }
    if (K == 0)
        alpha = 1.0f;   // the empty sum is +0 whatever alpha
    if (plan.config == kQ4Expanded) {
        if (K > 0 && launch_q4_expand((const uint32_t *)codes, (const uint32_t *)words, (_Float16 *)workspace, N, K, group,
                                      (hipStream_t)stream) != hipSuccess)
            return GEMM_F16_ERROR_LAUNCH_FAILED;
        return gemm_f16_scaled(M, N, K, A, 0, workspace, 1, C, alpha, epilogue, GEMM_F16_CONFIG_AUTO, stream);
    }
    Q4Args a;
    a.A = (const _Float16 *)A;
    a.codes = (const uint32_t *)codes;
    a.words = (const uint32_t *)words;
    a.C = (_Float16 *)C;
    a.M = (int)M;
    a.rows = (int)M;
    a.row0 = 0;
    a.N = (int)N;
    a.K = (int)K;
    a.n_blocks = (int)((N + 15) / 16);
    a.k_blocks = (int)((K + 127) / 128);
    a.tiles_m = (int)plan.tiles_m;
    a.tiles_n = (int)plan.tiles_n;
    a.splits = plan.splits;
    a.split_blocks = (int)plan.k_tiles;
    a.W = plan.splits > 1 ? (float *)workspace : nullptr;
    a.alpha = alpha;
    a.relu = epilogue == GEMM_F16_EPILOGUE_RELU ? 1 : 0;
    const hipError_t e = kQ4Configs[plan.config].stages == 0
                             ? launch_q4(plan.config, group, a, (hipStream_t)stream)
                             : launch_q4_tile(plan.config, group, a, plan.grid, (hipStream_t)stream);
    if (e != hipSuccess || plan.splits == 1)
        return status_of(e);
    return status_of(launch_reduce(a.W, a.C, M, N, plan.splits, a.alpha, a.relu, N % 4 == 0 && (uintptr_t)C % 8 == 0,
                                   (hipStream_t)stream));
}

gemm_f16_status_t gemm_f16_plan_q4(int64_t M, int64_t N, int64_t K, int group, const void *A, int config, int splits,
                                   gemm_f16_plan_t *plan)
{
    if (!plan || M < 0 || N < 0 || K < 0 || !known_group(group))
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (M > GEMM_F16_MAX_DIM || N > GEMM_F16_MAX_N || K > GEMM_F16_MAX_K)
        return GEMM_F16_ERROR_UNSUPPORTED_SIZE;
    return make_plan(M, N, K, group, rows_4_aligned(A, K), config, splits, plan);
}

int gemm_f16_q4_num_configs(void) { return kNumQ4Configs; }

const char *gemm_f16_q4_config_name(int config)
{
    if (config < 0 || config >= kNumQ4Configs)
        return nullptr;
    return kQ4Configs[config].name;
}

gemm_f16_status_t gemm_f16_q4_cache_append(const gemm_f16_q4_cache_t *cache, int64_t batch, int64_t tokens,
                                           int64_t max_pages, const void *K, int64_t k_stride, const void *V,
                                           int64_t v_stride, const int32_t *table, const int32_t *lengths,
                                           const int32_t *starts, const void *Q, int64_t q_stride, void *Q_out,
                                           int q_heads, const float *cos, const float *sin, int64_t positions,
                                           int rotary_dim, int interleaved, void *stream)
{
    gemm_f16_status_t st = validate_cache(cache, batch, max_pages);
    if (st != GEMM_F16_SUCCESS)
        return st;
    const int D = cache->head_dim;
    if (tokens < 0 || (!starts && tokens != batch) || !Q != !Q_out || (Q && q_heads < 1) || !cos != !sin ||
        (interleaved != 0 && interleaved != 1))
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (cos ? (positions < 0 || rotary_dim < 16 || rotary_dim > D || rotary_dim % 16 != 0) : rotary_dim != 0)
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (tokens > GEMM_F16_Q4_MAX_TOKENS || (Q && q_heads > GEMM_F16_Q4_MAX_HEADS))
        return GEMM_F16_ERROR_UNSUPPORTED_SIZE;
    if (tokens == 0 || batch == 0)
        return GEMM_F16_SUCCESS;
    if (!K || !V || !lengths || (max_pages > 0 && !table))
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (!rows_fit(k_stride, cache->heads, D) || !rows_fit(v_stride, cache->heads, D) || (Q && !rows_fit(q_stride, q_heads, D)))
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (!rows_reach(tokens, k_stride) || !rows_reach(tokens, v_stride) || (Q && !rows_reach(tokens, q_stride)) ||
        (cos && positions > kMostBytes / (2 * rotary_dim)))
        return GEMM_F16_ERROR_UNSUPPORTED_SIZE;
    if (((uintptr_t)K | (uintptr_t)V | (uintptr_t)Q | (uintptr_t)Q_out) & 1u ||
        ((uintptr_t)table | (uintptr_t)lengths | (uintptr_t)starts | (uintptr_t)cos | (uintptr_t)sin) & 3u)
        return GEMM_F16_ERROR_MISALIGNED;
    const int64_t width = (int64_t)cache->heads * D, q_width = (int64_t)q_heads * D, out_bytes = Q ? 2 * tokens * q_width : 0;
    const int64_t k_bytes = rows_bytes(tokens, k_stride, width), v_bytes = rows_bytes(tokens, v_stride, width);
    const bool in_place = Q && Q == Q_out && q_stride == q_width;
    const int64_t turn_bytes = cos ? positions * (rotary_dim / 2) * 4 : 0;
    if (!buffers_apart(cache) || overlaps_cache(K, k_bytes, cache) || overlaps_cache(V, v_bytes, cache) ||
        overlaps_cache(Q_out, out_bytes, cache) || overlaps_cache(table, batch * max_pages * 4, cache) ||
        overlaps_cache(lengths, batch * 4, cache) || (starts && overlaps_cache(starts, (batch + 1) * 4, cache)) ||
        (Q && overlaps_cache(Q, rows_bytes(tokens, q_stride, q_width), cache)) || overlaps_cache(cos, turn_bytes, cache) ||
        overlaps_cache(sin, turn_bytes, cache) || overlaps(Q_out, out_bytes, K, k_bytes) ||
        overlaps(Q_out, out_bytes, V, v_bytes) || overlaps(Q_out, out_bytes, cos, turn_bytes) ||
        overlaps(Q_out, out_bytes, sin, turn_bytes) || overlaps(Q_out, out_bytes, table, batch * max_pages * 4) ||
        overlaps(Q_out, out_bytes, lengths, batch * 4) || (starts && overlaps(Q_out, out_bytes, starts, (batch + 1) * 4)) ||
        (!in_place && Q && overlaps(Q_out, out_bytes, Q, rows_bytes(tokens, q_stride, q_width))))
        return GEMM_F16_ERROR_INVALID_VALUE;
    int dev = -1;
    st = check_device(&dev);
    if (st != GEMM_F16_SUCCESS)
        return st;
    Q4AppendArgs a;
    a.c = pages_of(cache, table, batch, max_pages);
    a.K = (const _Float16 *)K;
    a.V = (const _Float16 *)V;
    a.Q = (const _Float16 *)Q;
    a.Q_out = (_Float16 *)Q_out;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_stride = q_stride;
    a.lengths = lengths;
    a.starts = starts;
    a.cos = cos;
    a.sin = sin;
    a.positions = positions;
    a.tokens = (int)tokens;
    a.q_heads = Q ? q_heads : 0;
    a.rotary = rotary_dim;
    a.interleaved = interleaved;
    a.vec_k = rows_aligned(K, k_stride);
    a.vec_v = rows_aligned(V, v_stride);
    a.vec_q = rows_aligned(Q, q_stride);
    a.vec_out = (uintptr_t)Q_out % 16 == 0;
    return status_of(launch_q4_append(a, (hipStream_t)stream));
}

gemm_f16_status_t gemm_f16_q4_cache_read(const gemm_f16_q4_cache_t *cache, int64_t batch, int64_t tokens,
                                         int64_t max_pages, const int32_t *table, const int32_t *first,
                                         const int32_t *starts, void *K, void *V, void *stream)
{
    gemm_f16_status_t st = validate_cache(cache, batch, max_pages);
    if (st != GEMM_F16_SUCCESS)
        return st;
    if (tokens < 0)
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (tokens > GEMM_F16_Q4_MAX_TOKENS)
        return GEMM_F16_ERROR_UNSUPPORTED_SIZE;
    if (tokens == 0 || batch == 0)
        return GEMM_F16_SUCCESS;
    if (!K || !V || !starts || (max_pages > 0 && !table))
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (((uintptr_t)K | (uintptr_t)V) % 16 || ((uintptr_t)table | (uintptr_t)first | (uintptr_t)starts) & 3u)
        return GEMM_F16_ERROR_MISALIGNED;
    const int64_t bytes = 2 * tokens * cache->heads * cache->head_dim;
    for (const void *out : {K, V})
        if (overlaps_cache(out, bytes, cache) || overlaps(out, bytes, table, batch * max_pages * 4) ||
            overlaps(out, bytes, starts, (batch + 1) * 4) || (first && overlaps(out, bytes, first, batch * 4)))
            return GEMM_F16_ERROR_INVALID_VALUE;
    if (overlaps(K, bytes, V, bytes))
        return GEMM_F16_ERROR_INVALID_VALUE;
    int dev = -1;
    st = check_device(&dev);
    if (st != GEMM_F16_SUCCESS)
        return st;
    Q4ReadArgs a;
    a.c = pages_of(cache, table, batch, max_pages);
    a.first = first;
    a.starts = starts;
    a.K = (_Float16 *)K;
    a.V = (_Float16 *)V;
    a.tokens = (int)tokens;
    return status_of(launch_q4_read(a, (hipStream_t)stream));
}

gemm_f16_status_t gemm_f16_q4_attention(const gemm_f16_q4_cache_t *cache, int64_t batch, int q_heads, int64_t max_pages,
                                        const void *Q, int64_t q_stride, const int32_t *table, const int32_t *lengths,
                                        float scale, void *out, int splits, int64_t max_length, void *workspace,
                                        int64_t workspace_bytes, void *stream)
{
    gemm_f16_status_t st = validate_cache(cache, batch, max_pages);
    if (st != GEMM_F16_SUCCESS)
        return st;
    if (workspace_bytes < 0 || (!workspace && workspace_bytes != 0) || max_length < 0 || !std::isfinite(scale))
        return GEMM_F16_ERROR_INVALID_VALUE;
    const int64_t room = max_pages * cache->page_size;
    gemm_f16_plan_t plan;
    st = plan_attention(batch, q_heads, cache->heads, cache->head_dim, cache->group,
                        max_length > 0 ? std::min(max_length, room) : room, splits, &plan);
    if (st != GEMM_F16_SUCCESS)
        return st;
    if (batch == 0)
        return GEMM_F16_SUCCESS;
    const int64_t width = (int64_t)q_heads * cache->head_dim;
    if (!Q || !out || !lengths || (max_pages > 0 && !table) || (max_pages > 0 && cache->pages == 0) || q_stride < width)
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (!rows_reach(batch, q_stride))
        return GEMM_F16_ERROR_UNSUPPORTED_SIZE;
    if (!rows_aligned(Q, q_stride) || (uintptr_t)out % 16 || ((uintptr_t)table | (uintptr_t)lengths) & 3u)
        return GEMM_F16_ERROR_MISALIGNED;
    const int64_t out_bytes = 2 * batch * width, q_bytes = rows_bytes(batch, q_stride, width);
    if (overlaps(out, out_bytes, Q, q_bytes) || overlaps_cache(out, out_bytes, cache) ||
        overlaps(out, out_bytes, table, batch * max_pages * 4) || overlaps(out, out_bytes, lengths, batch * 4))
        return GEMM_F16_ERROR_INVALID_VALUE;
    if (plan.splits > 1) {
        if (!workspace)
            return GEMM_F16_ERROR_WORKSPACE;
        if ((uintptr_t)workspace % 16)
            return GEMM_F16_ERROR_MISALIGNED;
        if (workspace_bytes < plan.workspace_bytes)
            return GEMM_F16_ERROR_WORKSPACE;
        const int64_t wb = plan.workspace_bytes;
        if (overlaps(workspace, wb, Q, q_bytes) || overlaps(workspace, wb, out, out_bytes) ||
            overlaps_cache(workspace, wb, cache) || overlaps(workspace, wb, table, batch * max_pages * 4) ||
            overlaps(workspace, wb, lengths, batch * 4))
            return GEMM_F16_ERROR_INVALID_VALUE;
    }
    int dev = -1;
    st = check_device(&dev);
    if (st != GEMM_F16_SUCCESS)
        return st;
    Q4AttentionArgs a;
    a.c = pages_of(cache, table, batch, max_pages);
    a.Q = (const _Float16 *)Q;
    a.q_stride = q_stride;
    a.lengths = lengths;
    a.out = (_Float16 *)out;
    a.parts = plan.splits > 1 ? (float *)workspace : nullptr;
    a.scale = scale;
    a.q_heads = q_heads;
    a.ratio = q_heads / cache->heads;
    a.row_tiles = (a.ratio + 15) / 16;
    a.splits = plan.splits;
    a.step = plan.block_n;
    return status_of(launch_q4_attention(a, plan.grid, (hipStream_t)stream));
}

gemm_f16_status_t gemm_f16_plan_q4_attention(int64_t batch, int q_heads, int heads, int head_dim, int group,
                                             int64_t max_length, int splits, gemm_f16_plan_t *plan)
{
    if (!plan)
        return GEMM_F16_ERROR_INVALID_VALUE;
    return plan_attention(batch, q_heads, heads, head_dim, group, max_length, splits, plan);
}

} // extern "C"
