// gemm_f16_q4_attention.hip -- attention of one query token per sequence over
// the 4-bit paged cache.
//
// out[h] = sum_t softmax_t(scale q[h] . k[t]) v[t].  A workgroup owns up to 16
// query heads that share a cache head, and one part of a sequence's tokens;
// each of its waves takes every 4th step of SUB blocks of 32 tokens, keeps the
// running maximum m and sum l of the softmax and the unnormalised output in
// registers, and the waves' results are joined through LDS at the end.
//
// Scores: S^T = K Q^T with v_mfma_f32_16x16x32_f16, 16 tokens by 16 heads.
// Codes enter as 64 + q (exact, seven instructions a dword); the accumulator
// starts at -64 times the sum of the group's x, so that the product is
// sum q x, and the score the sum over groups of s (sum q x - z sum x), in fp32.
// The rows of the two 16-token products of a block are chosen so that lane
// (g, head) ends up with the scores of tokens 8 g .. 8 g + 7 of the block:
// row i of product u is token 8 (i / 4) + 4 u + i % 4.  That is the layout in
// which the probabilities enter the second product as its second operand, so
// they never leave the lane's registers.
//
// Output: O^T = V^T P^T, 16 values of d by 16 heads; the first operand's lane
// (g, d) takes tokens 8 g .. 8 g + 7 of one d, which is one dword of v_codes.
// A value's scale belongs to its token, the dimension that is summed over, so
// it multiplies the probability: P' = p s, one P' per group of d; q - z stays
// exact (and signed: an offset in it would cancel over all tokens).  P'
// enters as two binary16 parts (22 bits), so that the output carries no error
// beyond fp32's and its own rounding.
//
// Few heads (SUB 2 or 4): the 16 columns hold 16 / SUB heads SUB times, and the
// columns' copies take one block of the step each, so that scales, softmax
// and P', which a lane computes for its column, are computed once and not for
// columns that nobody asked for.  Scores of a block are kept by its own columns;
// P' of the others is zero in its second product, whose sums thus stay apart:
// every column is a softmax of its own until the join.  The values' zero
// points, which a lane has for its own block, go to the row's other lanes by
// broadcast.  Of about 400 vector instructions for 32 tokens (head_dim 128,
// groups of 64) 240 remain with SUB 4.
//
// p = exp2(x - base), where base is chosen so that P' stays inside binary16:
// when a step's largest score plus log2 of its largest scale passes base by
// more than 15, base moves to 12 below it and the sums are rescaled; between,
// nothing is (3 bits of slack make that rare).  The two may be different tokens',
// so where scales of a step differ by more than 5 bits, base moves no further
// than 6 below the largest p s of any token so far: a large value without weight
// takes no bits from the others.  A group of d whose own largest p s lies more than
// 8 bits below 2^12 is lifted by a power of two of its own, taken off its sums at the
// end, so that its outputs lose none to another group's scale.  So every group's
// largest P' is between 2^3 and 2^15, and all are exact to 2^-24.  From scores of 2^23
// on, whose rounding reaches whole powers of two, base is the largest score itself,
// rounded as the scores are: tokens that share it share the weight, with P' = s.
// The sums of p and of P' v carry the same factor 2^-base, which the quotient drops.
//
// Scales of like size skip the tokens' own p s: taken in every wave's first step
// they cost 0.3 us of 3.7 for one sequence of 100 and 2 of 27 for 32 x 4096.  And
// nothing of this is held in registers, where largest[] costs 2 of 27 us, but in LDS.
#include <type_traits>

#include "gemm_f16_q4.h"
#include "gemm_f16_q4_format.h"
#include "gemm_f16_tile.h"

namespace gemm_f16_impl {

constexpr int WAVES = kQ4AttentionWaves, BLOCK = kQ4AttentionTokens;
constexpr float kLog2e = 1.4426950408889634f;

constexpr float kTop = 15.0f, kLift = 12.0f;   // P' stays below 2^kTop and starts below 2^kLift
constexpr float kLoose = 6.0f;                 // bits that the bound on P' may exceed their largest by, when base moves
constexpr float kApart = 8.0f;                 // bits between groups of d that share their powers of two
constexpr float kFar = 0x1p23f;                // scores whose rounding reaches whole powers of two
constexpr float kNone = -0x1p126f;             // base without a token: exp2(kNone) is 0, exp2(-kNone) infinite

// Waves of a SIMD the registers are shared out to: as many as leave the sums,
// a step's codes and words and the products' operands in registers (groups of
// 128 would fit 3 times, and take 33.5 us for one sequence of 131000 then, not 32.7).
// Waves that take turns serve better than a wave that loads ahead: with the
// next step's keys on their way during the softmax and its values during the
// next scores, in the same registers but for the addresses', 32 x 4096 tokens
// of groups of 64 take 29 us, not 26.2, and of 128 27.2, not 24.4; only one sequence
// of 131000 is hardly slower so.  Page lookups for every 8 tokens and four blocks
// side by side do not fit with groups of 64 3 times: with 44 bytes of a lane in
// scratch, 32 x 4096 tokens in pages of 16 take 34.4 us, not 31.5, and 64 x 4000 59.7, not 49.4.
constexpr int attention_waves(int head_dim, int group, int sub, bool one)
{
    if (head_dim == 128 && group == 64 && sub == 4 && !one)
        return 2;
    return head_dim == 256 ? (group < 128 ? 1 : 2) : head_dim == 128 && group != 64 ? 2 : 3;
}

// Steps of a part: whole turns of the workgroup's waves.
__device__ __forceinline__ int part_steps(int steps, int splits)
{
    return ((steps + splits - 1) / splits + WAVES - 1) / WAVES * WAVES;
}

// Two values rounded towards zero to binary16, packed.  Only for splitting a
// value into two parts: the second takes up what the first leaves.
__device__ __forceinline__ q4_half2 pack_rtz(float a, float b)
{
    return __builtin_bit_cast(q4_half2, __builtin_amdgcn_cvt_pkrtz(a, b));
}

// v / total as four binary16; zeros where there are no tokens (NaN stays).
__device__ __forceinline__ void store_quotient(half_t *to, const float4v &v, float total)
{
    const float inv = total > 0.0f ? 1.0f / total : total == 0.0f ? 0.0f : total;
    half4 out;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        out[r] = (half_t)(v[r] * inv);
    *reinterpret_cast<half4 *>(to) = out;
}

// Maximum (or sum) over the four lanes that share a column: lanes 16 and 32
// apart.  The swaps exchange rows of 16 or halves of 32 lanes between two
// registers; of two copies of x they leave each pair's values side by side.
__device__ __forceinline__ float column_max(float x)
{
    const unsigned v = __builtin_bit_cast(unsigned, x);
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    x = __builtin_fmaxf(__builtin_bit_cast(float, (unsigned)a[0]), __builtin_bit_cast(float, (unsigned)a[1]));
    const unsigned w = __builtin_bit_cast(unsigned, x);
    const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    return __builtin_fmaxf(__builtin_bit_cast(float, (unsigned)b[0]), __builtin_bit_cast(float, (unsigned)b[1]));
}
__device__ __forceinline__ float column_sum(float x)
{
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// The value of lane LANE of each row of 16 lanes, in all of them.
template <int LANE>
__device__ __forceinline__ unsigned row_lane(unsigned x)
{
    return (unsigned)__builtin_amdgcn_mov_dpp((int)x, 0x150 + LANE, 0xF, 0xF, true);   // row_newbcast
}

// What a wave needs of SUB blocks of 32 tokens, in the layout of its products;
// the words are those of the lane's own block.
template <int D, int GROUP, int SUB>
struct AttentionStep {
    static constexpr int GROUPS = D / GROUP;
    unsigned k[SUB][2][D / 32];     // codes of token 8 (col / 4) + 4 u + col % 4
    uint4 k_words[2][GROUPS];       // of tokens 8 g + 4 u .. + 3
    uint4 v_words[2][GROUPS];
    unsigned v[SUB][D / 16];        // d = 16 i + col of tokens 8 g .. + 7
};

// Where they lie: pages of the blocks (of this lane's granules of 8 tokens,
// for a row of K and for the values, without ONE) and of the lane's words.
template <int SUB>
struct AttentionPages {
    int k[SUB], v[SUB], own;
};

// ONE: every block of 32 tokens lies in one page (page sizes that are
// multiples of 32): the page is the wave's and addresses are scalar, but for
// each lane's place in the block.  Else pages are looked up for every granule
// of 8 tokens.
template <int D, int GROUP, int SUB, bool ONE>
__global__ void __launch_bounds__(64 * WAVES, attention_waves(D, GROUP, SUB, ONE)) q4_attention_kernel(Q4AttentionArgs a)
{
    constexpr int GROUPS = D / GROUP, JG = GROUP / 32, TILES = D / 16, PITCH = D + 4;
    constexpr int HEADS = 16 / SUB, STEP = BLOCK * SUB;
    extern __shared__ __attribute__((aligned(16))) unsigned char q4_attention_lds[];
    float *sums = reinterpret_cast<float *>(q4_attention_lds);   // [wave][16 columns][PITCH]
    float *stats = sums + WAVES * 16 * PITCH;                    // [wave][base, l][16 columns]

    const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, g = lane >> 4, own = col / HEADS;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // heads first, so that the XCDs (workgroups in turn) get equal work; parts
    // last, so that the sequences' first ones, which are whole, start first
    unsigned id = blockIdx.x;
    const int h = id % a.c.heads;
    id /= a.c.heads;
    const int tile = id % a.row_tiles;
    id /= a.row_tiles;
    const int b = id % a.c.batch, split = id / a.c.batch;
    const int rows = min(a.ratio - HEADS * tile, HEADS);         // query heads of this workgroup
    const int64_t q_head = (int64_t)h * a.ratio + HEADS * tile;

    // this lane's head of Q, elements 32 j + 8 g .. + 7
    half8 q[D / 32];
    const half_t *query = a.Q + b * a.q_stride + (q_head + min(col % HEADS, rows - 1)) * D + 8 * g;
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
        q[j] = *reinterpret_cast<const half8 *>(query + 32 * j);

    const int length = __builtin_amdgcn_readfirstlane(
        (int)min((int64_t)max(a.lengths[b], 0), (int64_t)a.c.max_pages * a.c.page_size));
    const int steps = (length + STEP - 1) / STEP, per = part_steps(steps, a.splits);
    const int first = split * per, last = min(steps, first + per);
    if (first >= last && (a.splits > 1 || length > 0))
        return;                                                  // an empty part; the join does not read it

    // Reads stay inside the sequence's row of the table whatever the step.
    const int32_t *table = a.c.table + (int64_t)b * a.c.max_pages;
    const auto page_at = [&](int token) { return table[min(q4_page_of(a.c, token), a.c.max_pages - 1)]; };
    // This lane's place in a block: as a row of K, and as holder of 8 tokens
    const int k_token = 8 * (col / 4) + (col & 3), g_token = 8 * g;
    typedef AttentionPages<SUB> Pages;
    const auto next_pages = [&](int step, Pages &p) {
        const int t0 = step * STEP;
#pragma unroll
        for (int i = 0; i < SUB; ++i) {
            if constexpr (ONE) {
                p.k[i] = page_at(t0 + BLOCK * i);
            } else {
                p.k[i] = page_at(t0 + BLOCK * i + 8 * (col / 4));
                p.v[i] = page_at(t0 + BLOCK * i + g_token);
            }
        }
        if constexpr (SUB > 1)
            p.own = page_at(t0 + BLOCK * own + g_token);
        else
            p.own = ONE ? p.k[0] : p.v[0];
    };
    const auto exists = [&](int page) { return page >= 0 && page < a.c.pages; };
    // A block's codes and words come from page 0 where there is no page.
    typedef AttentionStep<D, GROUP, SUB> Step;
    const auto load_words = [&](int step, const Pages &p, const uint32_t *words, uint4 (&w)[2][GROUPS]) {
        const int t = step * STEP + BLOCK * own + g_token;
        const int64_t hp = (int64_t)(exists(p.own) ? p.own : 0) * a.c.heads + h;
        const uint32_t *from = words + hp * GROUPS * a.c.page_size + (t - q4_page_of(a.c, t) * a.c.page_size);
#pragma unroll
        for (int n = 0; n < GROUPS; ++n)
#pragma unroll
            for (int u = 0; u < 2; ++u)
                w[u][n] = *reinterpret_cast<const uint4 *>(from + n * a.c.page_size + 4 * u);
    };
    const auto load_k = [&](int step, const Pages &p, Step &x) {
#pragma unroll
        for (int i = 0; i < SUB; ++i) {
            const uint32_t *kc;
            if constexpr (ONE) {
                const int page = __builtin_amdgcn_readfirstlane(p.k[i]), t = step * STEP + BLOCK * i;
                const int64_t hp = (int64_t)(exists(page) && t < length ? page : 0) * a.c.heads + h;
                const int slot = t - q4_page_of(a.c, t) * a.c.page_size;
                kc = a.c.k_codes + (hp * a.c.page_size + slot) * (D / 8) + k_token * (D / 8);
            } else {
                const int t = step * STEP + BLOCK * i + 8 * (col / 4);
                const int64_t hp = (int64_t)(exists(p.k[i]) && t < length ? p.k[i] : 0) * a.c.heads + h;
                const int slot = t - q4_page_of(a.c, t) * a.c.page_size + (col & 3);
                kc = a.c.k_codes + (hp * a.c.page_size + slot) * (D / 8);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if constexpr (D == 64) {
                    const uint2 v = *reinterpret_cast<const uint2 *>(kc + u * (4 * D / 8) + 2 * g);
                    x.k[i][u][0] = v.x;
                    x.k[i][u][1] = v.y;
                } else {
#pragma unroll
                    for (int n = 0; n < D / 128; ++n) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(kc + u * (4 * D / 8) + 16 * n + 4 * g);
                        x.k[i][u][4 * n] = v.x;
                        x.k[i][u][4 * n + 1] = v.y;
                        x.k[i][u][4 * n + 2] = v.z;
                        x.k[i][u][4 * n + 3] = v.w;
                    }
                }
            }
        }
        load_words(step, p, a.c.k_words, x.k_words);
    };
    const auto load_v = [&](int step, const Pages &p, Step &x) {
        load_words(step, p, a.c.v_words, x.v_words);
#pragma unroll
        for (int i = 0; i < SUB; ++i) {
            const uint32_t *vc;
            if constexpr (ONE) {
                const int page = __builtin_amdgcn_readfirstlane(p.k[i]), t = step * STEP + BLOCK * i;
                const int64_t hp = (int64_t)(exists(page) && t < length ? page : 0) * a.c.heads + h;
                const int slot = t - q4_page_of(a.c, t) * a.c.page_size;
                vc = a.c.v_codes + (hp * (a.c.page_size / 8) + slot / 8) * D + (g * 16 + col) * TILES;
            } else {
                const int t = step * STEP + BLOCK * i + g_token;
                const int64_t hp = (int64_t)(exists(p.v[i]) && t < length ? p.v[i] : 0) * a.c.heads + h;
                const int slot = t - q4_page_of(a.c, t) * a.c.page_size;
                vc = a.c.v_codes + (hp * (a.c.page_size / 8) + slot / 8) * D + col * TILES;
            }
#pragma unroll
            for (int e = 0; e < TILES; e += 4) {
                const uint4 v = *reinterpret_cast<const uint4 *>(vc + e);
                x.v[i][e] = v.x;
                x.v[i][e + 1] = v.y;
                x.v[i][e + 2] = v.z;
                x.v[i][e + 3] = v.w;
            }
        }
    };

    // The sign of the scale goes into the queries (exactly), so that the
    // largest product is the largest score.
    const float scale = __builtin_fmaxf(__builtin_fabsf(a.scale) * kLog2e, 0x1p-126f);   // 0 would undo -infinity
    float q_sum[GROUPS];
    float4v start[GROUPS];         // takes the 64 off again
    const auto sum_queries = [&]() {
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
            q[j] = a.scale < 0.0f ? -q[j] : q[j];
#pragma unroll
        for (int n = 0; n < GROUPS; ++n) {
            float t = 0.0f;
#pragma unroll
            for (int j = n * JG; j < (n + 1) * JG; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    t += (float)q[j][i];
            q_sum[n] = column_sum(t);
            const float off = -64.0f * q_sum[n];
            start[n] = float4v{off, off, off, off};
        }
    };
    const q4_bits bits;

    float base = kNone, l = 0.0f;
    // log2 of the largest p s of each group so far, rounded up, is at least base +
    // kLift - kLoose; once scales have differed by more it is kept where the sums
    // will go, [group][column]
    float *const largest = sums + wave * 16 * PITCH + col;
    bool uneven = false, lifted = false, far = false;
    // 2^exponent(s) is more than |s|, twice that at most; 0 counts as the smallest
    const auto exponent = [](float v) { return v == 0.0f ? -23.0f : (float)__builtin_amdgcn_frexp_expf(v); };
    // log2 of the power of two that lifts a group
    const auto lift = [](float b, float most) {
        if constexpr (GROUPS == 1)
            return 0.0f;
        const float below = b + kLift - most;
        return below > kApart && __builtin_fabsf(b) < kFar ? __builtin_floorf(below) : 0.0f;
    };
    float4v acc[TILES];
#pragma unroll
    for (int i = 0; i < TILES; ++i)
        acc[i] = float4v{0, 0, 0, 0};

    // score / scale of the lane's tokens 8 g + 4 u + r of its own block
    const auto scores = [&](const Step &y, float (&x)[8]) {
#pragma unroll
        for (int n = 0; n < GROUPS; ++n)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float4v s;
#pragma unroll
                for (int i = 0; i < SUB; ++i) {
                    float4v t = start[n];
#pragma unroll
                    for (int j = n * JG; j < (n + 1) * JG; ++j)
                        t = __builtin_amdgcn_mfma_f32_16x16x32_f16(q4_codes_64(y.k[i][u][j], bits), q[j], t, 0, 0, 0);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        s[r] = i == 0 || own == i ? t[r] : s[r];
                }
                const uint4 w = y.k_words[u][n];
                const unsigned word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float t = __builtin_fmaf(-(float)(word[r] >> 16), q_sum[n], s[r]);
                    x[4 * u + r] = n == 0 ? q4_scale(word[r]) * t : __builtin_fmaf(q4_scale(word[r]), t, x[4 * u + r]);
                }
            }
    };
    const auto attend = [&](int step, const Pages &p, const Step &y, float (&x)[8]) __attribute__((always_inline)) {
        const int tg = step * STEP + BLOCK * own + g_token;
        const bool mine = exists(p.own);
        unsigned word[GROUPS][8];
#pragma unroll
        for (int n = 0; n < GROUPS; ++n) {
            const uint4 w0 = y.v_words[0][n], w1 = y.v_words[1][n];
            const unsigned w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                word[n][i] = w[i];
        }
        if (!__all(mine && tg + 8 <= length)) {
            // what lies behind the last token has no weight, whatever it is, and
            // a word that is held anyway: of the lane's first token, or 0 without one
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool there = mine && tg + i < length;
                x[i] = there ? x[i] : -INFINITY;
#pragma unroll
                for (int n = 0; n < GROUPS; ++n)
                    word[n][i] = there ? word[n][i] : i == 0 ? 0u : word[n][0];
            }
        }
        // (the empty asm keeps one conversion of each scale for both uses;
        // the compiler would make a second one for the absolute value)
        float s[GROUPS][8];
#pragma unroll
        for (int n = 0; n < GROUPS; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[n][i] = q4_scale(word[n][i]);
                asm("" : "+v"(s[n][i]));
            }
        float most = x[0], top = 0.0f;
#pragma unroll
        for (int i = 1; i < 8; ++i)
            most = __builtin_fmaxf(most, x[i]);
#pragma unroll
        for (int n = 0; n < GROUPS; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                top = __builtin_fmaxf(top, __builtin_fabsf(s[n][i]));
        const bool some = most != -INFINITY;
        most = column_max(most);
        top = column_max(top);
        // no P' of the step passes this place
        const float reach = __builtin_fmaf(most, scale, exponent(top));
        const bool grown = reach > base + kTop;
        if (lifted || far || __any(grown)) {
            // scales within 5 bits of each other: every group has a p s of this size
            float least = top;
#pragma unroll
            for (int n = 0; n < GROUPS; ++n)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    least = __builtin_fminf(least, __builtin_fabsf(s[n][i]));
            const bool even = !some || least * 32.0f >= top;
            // where 12 is lost in the score's rounding, base is the score itself
            float peak_score = most * scale;
            asm("" : "+v"(peak_score));   // (not contracted with what follows)
            const bool beyond = __builtin_fabsf(peak_score) >= kFar;
            float to = beyond ? __builtin_fmaxf(base, peak_score) : grown ? reach - kLift : base, f[GROUPS];
            if (__builtin_expect(!uneven && __all(even || !grown), 1)) {
#pragma unroll
                for (int n = 0; n < GROUPS; ++n)
                    f[n] = 1.0f;
            } else {
                // each token's own p s, of the columns that moved or hold a lifted group
                const bool all_even = column_max(even ? 0.0f : 1.0f) == 0.0f;
                float most_of[GROUPS], peak = kNone;
                bool mine = grown, any = false;
#pragma unroll
                for (int n = 0; n < GROUPS; ++n) {
                    most_of[n] = uneven ? largest[16 * n] : base + (kLift - kLoose);
                    f[n] = lift(base, most_of[n]);
                    mine |= f[n] > 0.0f;
                }
#pragma unroll
                for (int n = 0; n < GROUPS; ++n) {
                    float r = kNone;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        r = __builtin_fmaxf(r, __builtin_fmaf(x[i], scale, exponent(s[n][i])));
                    r = column_max(r);
                    // (a lifted group's must not be passed; else as above, whatever the other columns do)
                    r = all_even && f[n] == 0.0f ? reach - kLoose : r;
                    most_of[n] = mine ? __builtin_fmaxf(most_of[n], r) : most_of[n];
                    peak = __builtin_fmaxf(peak, most_of[n]);
                    largest[16 * n] = most_of[n];
                }
                q4_wave_fence();
                to = beyond ? to : __builtin_fmaxf(base, __builtin_fminf(to, peak + (kLoose - kLift)));
#pragma unroll
                for (int n = 0; n < GROUPS; ++n) {
                    const float now = lift(to, most_of[n]), up = __builtin_amdgcn_exp2f(now);
                    any |= now > 0.0f;
                    f[n] = __builtin_amdgcn_exp2f(now - f[n]);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        s[n][i] *= up;
                }
                uneven = true;
                lifted = __any(any);
            }
            const float fade = __builtin_amdgcn_exp2f(base - to);
            base = to;
            far = __any(__builtin_fabsf(base) >= kFar && base > kNone);
            l *= fade;
#pragma unroll
            for (int n = 0; n < GROUPS; ++n) {
                f[n] *= fade;
#pragma unroll
                for (int i = n * GROUP / 16; i < (n + 1) * GROUP / 16; ++i)
                    acc[i] *= f[n];
            }
        }
        if (__builtin_expect(far, 0)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float t = x[i] * scale;
                asm("" : "+v"(t));
                const float d = __builtin_fabsf(base) >= kFar ? t - base : __builtin_fmaf(x[i], scale, -base);
                x[i] = __builtin_amdgcn_exp2f(d);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], scale, -base));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            l += x[i];
#pragma unroll
        for (int n = 0; n < GROUPS; ++n) {
            const unsigned *w = word[n];
            half8 hi, lo;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float p0 = x[i] * s[n][i], p1 = x[i + 1] * s[n][i + 1];
                const q4_half2 v = pack_rtz(p0, p1), rest = pack_rtz(p0 - (float)v[0], p1 - (float)v[1]);
                hi[i] = v[0];
                hi[i + 1] = v[1];
                lo[i] = rest[0];
                lo[i + 1] = rest[1];
            }
            const unsigned z[4] = {q4_zero(w[0] >> 16, w[1] >> 16).a, q4_zero(w[2] >> 16, w[3] >> 16).b,
                                   q4_zero(w[4] >> 16, w[5] >> 16).a, q4_zero(w[6] >> 16, w[7] >> 16).b};
            const auto block = [&](auto sub) {
                constexpr int i = decltype(sub)::value;
                // the other columns' tokens are not of this block
                uint4 hb = __builtin_bit_cast(uint4, hi), lb = __builtin_bit_cast(uint4, lo);
                unsigned zb[4] = {z[0], z[1], z[2], z[3]};
                if constexpr (SUB > 1) {
                    const unsigned keep = own == i ? ~0u : 0u;
                    hb = make_uint4(hb.x & keep, hb.y & keep, hb.z & keep, hb.w & keep);
                    lb = make_uint4(lb.x & keep, lb.y & keep, lb.z & keep, lb.w & keep);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        zb[k] = row_lane<i * HEADS>(zb[k]);
                }
#pragma unroll
                for (int e = n * GROUP / 16; e < (n + 1) * GROUP / 16; ++e) {
                    const half8 v = q4_codes(y.v[i][e], bits, zb[0], zb[1], zb[2], zb[3]);
                    acc[e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, __builtin_bit_cast(half8, hb), acc[e], 0, 0, 0);
                    acc[e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, __builtin_bit_cast(half8, lb), acc[e], 0, 0, 0);
                }
            };
            block(std::integral_constant<int, 0>{});
            if constexpr (SUB > 1)
                block(std::integral_constant<int, 1>{});
            if constexpr (SUB > 2) {
                block(std::integral_constant<int, 2>{});
                block(std::integral_constant<int, 3>{});
            }
        }
    };

    int step = first + wave;
    if (step < last) {
        // A step's pages are looked up before the loads of the step before it
        // go out: waiting for the pages must not wait for those.
        Pages here, next;
        Step y;
        float x[8];
        next_pages(step, here);
        sum_queries();
        for (; step < last; step += WAVES) {
            load_k(step, here, y);
            load_v(step, here, y);
            next_pages(step + WAVES, next);
            scores(y, x);
            attend(step, here, y, x);
            here = next;
        }
    }
    l = column_sum(l);
    if (lifted) {
#pragma unroll
        for (int n = 0; n < GROUPS; ++n) {
            const float f = __builtin_amdgcn_exp2f(-lift(base, largest[16 * n]));
#pragma unroll
            for (int i = n * GROUP / 16; i < (n + 1) * GROUP / 16; ++i)
                acc[i] *= f;
        }
        q4_wave_fence();
    }

    // join the waves and their columns: lane (g, col) holds d = 16 i + 4 g + r
#pragma unroll
    for (int i = 0; i < TILES; ++i)
        *reinterpret_cast<float4v *>(sums + (wave * 16 + col) * PITCH + 16 * i + 4 * g) = acc[i];
    if (g == 0) {
        stats[wave * 32 + col] = base;
        stats[wave * 32 + 16 + col] = l;
    }
    __syncthreads();
    for (int e = tid; e < rows * (D / 4); e += 64 * WAVES) {
        const int row = e / (D / 4), d = e % (D / 4) * 4;
        float top = kNone, total = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES * SUB; ++w)
            top = __builtin_fmaxf(top, stats[w / SUB * 32 + w % SUB * HEADS + row]);
        float4v v = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < WAVES * SUB; ++w) {
            const int at = w % SUB * HEADS + row;
            const float f = __builtin_amdgcn_exp2f(stats[w / SUB * 32 + at] - top);
            total += f * stats[w / SUB * 32 + 16 + at];
            const float4v part = *reinterpret_cast<const float4v *>(sums + (w / SUB * 16 + at) * PITCH + d);
            v += f * part;
        }
        const int64_t head = (int64_t)b * a.q_heads + q_head + row;
        if (a.splits == 1) {
            store_quotient(a.out + head * D + d, v, total);
        } else {
            *reinterpret_cast<float4v *>(a.parts + (head * a.splits + split) * D + d) = v;
            if (d == 0) {
                float2 *ml = reinterpret_cast<float2 *>(a.parts + (int64_t)a.c.batch * a.q_heads * a.splits * D);
                ml[head * a.splits + split] = make_float2(top, total);
            }
        }
    }
}

constexpr int FEW = 8;

// Join the parts of the heads: D / 4 lanes hold a head's elements, and TEAMS
// teams of them take its parts in turn; the teams' sums are added in order.
// With one team a workgroup joins several heads, of
// at most FEW parts each.
template <int D, int TEAMS>
__global__ void __launch_bounds__(256) q4_attention_join_kernel(Q4AttentionArgs a)
{
    constexpr int LANES = D / 4, HEADS = 256 / LANES / TEAMS;
    static_assert(TEAMS == 1 || HEADS == 1, "several heads, or several teams");
    __shared__ float4v sums[TEAMS][HEADS * LANES];
    __shared__ float totals[TEAMS][HEADS];
    const int d = threadIdx.x % LANES, team = threadIdx.x / LANES % TEAMS, mine = threadIdx.x / (LANES * TEAMS);
    const int64_t heads = (int64_t)a.c.batch * a.q_heads, head = (int64_t)blockIdx.x * HEADS + mine;
    float total = 0.0f;
    float4v v = {0, 0, 0, 0};
    if (head < heads) {
        const float2 *ml = reinterpret_cast<const float2 *>(a.parts + heads * a.splits * D) + head * a.splits;
        const float *part = a.parts + head * a.splits * D + 4 * d;
        const int length = (int)min((int64_t)max(a.lengths[head / a.q_heads], 0), (int64_t)a.c.max_pages * a.c.page_size);
        const int steps = (length + a.step - 1) / a.step, per = part_steps(steps, a.splits);
        const int used = per > 0 ? (steps + per - 1) / per : 0;      // parts that hold tokens
        const auto add = [&](float base, const float2 &w, const float4v &x) {
            const float f = __builtin_amdgcn_exp2f(w.x - base);
            total += f * w.y;
            v += f * x;
        };
        float top = kNone;
        if constexpr (TEAMS > 1) {   // one head: every wave looks at all parts
            for (int s = threadIdx.x & 63; s < used; s += 64)
                top = __builtin_fmaxf(top, ml[s].x);
#pragma unroll
            for (int m = 1; m < 64; m *= 2)
                top = __builtin_fmaxf(top, __shfl_xor(top, m));
#pragma unroll 4
            for (int s = team; s < used; s += TEAMS)
                add(top, ml[s], *reinterpret_cast<const float4v *>(part + s * D));
        } else {
            // all parts are read at once, whether the length says that they
            // are used or not: 0.5 us less than one read after the other
            float4v x[FEW];
            float2 w[FEW];
#pragma unroll
            for (int i = 0; i < FEW; ++i) {
                const int s = min(i, a.splits - 1);
                x[i] = *reinterpret_cast<const float4v *>(part + s * D);
                w[i] = ml[s];
            }
#pragma unroll
            for (int i = 0; i < FEW; ++i)
                top = i < used ? __builtin_fmaxf(top, w[i].x) : top;
#pragma unroll
            for (int i = 0; i < FEW; ++i)
                if (i < used)
                    add(top, w[i], x[i]);
        }
    }
    if constexpr (TEAMS > 1) {
        sums[team][mine * LANES + d] = v;
        if (d == 0)
            totals[team][mine] = total;
        __syncthreads();
        if (team > 0)
            return;
#pragma unroll
        for (int t = 1; t < TEAMS; ++t) {
            v += sums[t][mine * LANES + d];
            total += totals[t][mine];
        }
    }
    if (head < heads)
        store_quotient(a.out + head * D + 4 * d, v, total);
}

int64_t q4_attention_lds_bytes(int head_dim) { return 4 * WAVES * (16 * (head_dim + 4) + 32); }

template <int D, int GROUP, int SUB>
static void launch_parts(const Q4AttentionArgs &a, int64_t grid, hipStream_t s)
{
    if (a.c.page_size % BLOCK == 0)
        hipLaunchKernelGGL((q4_attention_kernel<D, GROUP, SUB, true>), dim3((unsigned)grid), dim3(64 * WAVES),
                           (unsigned)q4_attention_lds_bytes(D), s, a);
    else
        hipLaunchKernelGGL((q4_attention_kernel<D, GROUP, SUB, false>), dim3((unsigned)grid), dim3(64 * WAVES),
                           (unsigned)q4_attention_lds_bytes(D), s, a);
}

template <int D, int GROUP>
static hipError_t launch_attention(const Q4AttentionArgs &a, int64_t grid, hipStream_t s)
{
    if (a.step == BLOCK)
        launch_parts<D, GROUP, 1>(a, grid, s);
    else if (a.step == 2 * BLOCK)
        launch_parts<D, GROUP, 2>(a, grid, s);
    else if (D < 256)
        launch_parts<D, GROUP, D < 256 ? 4 : 1>(a, grid, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1)
        return e;
    // few parts: a team for each head; many: all of a workgroup's teams
    const int64_t heads = (int64_t)a.c.batch * a.q_heads;
    constexpr int TEAMS = 1024 / D;
    if (a.splits <= FEW)
        hipLaunchKernelGGL((q4_attention_join_kernel<D, 1>), dim3((unsigned)((heads + TEAMS - 1) / TEAMS)), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((q4_attention_join_kernel<D, TEAMS>), dim3((unsigned)heads), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_q4_attention(const Q4AttentionArgs &a, int64_t grid, hipStream_t s)
{
    switch (a.c.head_dim * 1000 + a.c.group) {
    case 64032: return launch_attention<64, 32>(a, grid, s);
    case 64064: return launch_attention<64, 64>(a, grid, s);
    case 128032: return launch_attention<128, 32>(a, grid, s);
    case 128064: return launch_attention<128, 64>(a, grid, s);
    case 128128: return launch_attention<128, 128>(a, grid, s);
    case 256032: return launch_attention<256, 32>(a, grid, s);
    case 256064: return launch_attention<256, 64>(a, grid, s);
    case 256128: return launch_attention<256, 128>(a, grid, s);
    default: return hipErrorInvalidValue;
    }
}

} // namespace gemm_f16_impl
