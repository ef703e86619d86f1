// gemm_f16_q4_attention.hip -- attention of one query token per sequence over
// the 4-bit paged cache.
//
// out[h] = sum_t softmax_t(scale q[h] . k[t]) v[t].  A workgroup owns up to 16
// query heads that share a cache head, and one part of a sequence's tokens;
// each of its waves takes every 4th block of 32 tokens, keeps the running
// maximum m and sum l of the softmax and the unnormalised output in
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
// p = exp2(x - base), where base is chosen so that P' stays inside binary16:
// when a block's largest score plus log2 of its largest scale passes base by
// more than 15, base moves to 12 below it and the sums are rescaled; between,
// nothing is (3 bits of slack make that rare).  So P' is below 2^15 and exact
// to 2^-24, 2^-36 of the largest.  The sums of p and of P' v carry the same
// factor, which the quotient drops.
#include "gemm_f16_q4_format.h"
#include "gemm_f16_tile.h"

namespace gemm_f16_impl {

constexpr int WAVES = kQ4AttentionWaves, STEP = kQ4AttentionTokens;
constexpr float kLog2e = 1.4426950408889634f;

constexpr float kTop = 15.0f, kLift = 12.0f;   // P' stays below 2^kTop and starts below 2^kLift

// Waves of a SIMD the registers are shared out to.  At 32 x 4096 tokens,
// head_dim 128: group 64 30.1 us with 2 (and a block's loads ahead), 28.1 with 3
// (without); group 128 25.9 with 2, 27.0 with 3, and 32.9 against 37.3 for one
// sequence of 131000.
constexpr int attention_waves(int head_dim, int group)
{
    return head_dim == 256 ? (group < 128 ? 1 : 2) : head_dim / group == 1 ? 2 : 3;
}

// Blocks of a part: whole turns of the workgroup's waves.
__device__ __forceinline__ int part_blocks(int blocks, int splits)
{
    return ((blocks + splits - 1) / splits + WAVES - 1) / WAVES * WAVES;
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

// What a wave needs of 32 tokens, in the layout of its products.
template <int D, int GROUP>
struct AttentionBlock {
    static constexpr int GROUPS = D / GROUP, REGISTERS = D / 8 + 16 * GROUPS;
    unsigned k[2][D / 32];          // codes of token 8 (col / 4) + 4 u + col % 4
    uint4 k_words[2][GROUPS];       // of tokens 8 g + 4 u .. + 3
    uint4 v_words[2][GROUPS];
    unsigned v[D / 16];             // d = 16 i + col of tokens 8 g .. + 7
    bool mine;                      // the page of tokens 8 g .. exists
    int whole;                      // all 32 tokens do
};

// ONE: every block of 32 tokens lies in one page (page sizes that are
// multiples of 32): the page is the wave's and addresses are scalar, but for
// each lane's place in the block.  Else pages are looked up for every granule
// of 8 tokens.
template <int D, int GROUP, bool ONE>
__global__ void __launch_bounds__(64 * WAVES, attention_waves(D, GROUP)) q4_attention_kernel(Q4AttentionArgs a)
{
    constexpr int GROUPS = D / GROUP, JG = GROUP / 32, BLOCKS = D / 16, PITCH = D + 4;
    extern __shared__ __attribute__((aligned(16))) unsigned char q4_attention_lds[];
    float *sums = reinterpret_cast<float *>(q4_attention_lds);   // [wave][16 heads][PITCH]
    float *stats = sums + WAVES * 16 * PITCH;                    // [wave][base, l][16 heads]

    const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int id = blockIdx.x;
    const int split = id % a.splits;
    id /= a.splits;
    const int tile = id % a.row_tiles;
    id /= a.row_tiles;
    const int h = id % a.c.heads, b = id / a.c.heads;
    const int rows = min(a.ratio - 16 * tile, 16);               // query heads of this workgroup
    const int64_t q_head = (int64_t)h * a.ratio + 16 * tile;

    const int length = __builtin_amdgcn_readfirstlane(
        (int)min((int64_t)max(a.lengths[b], 0), (int64_t)a.c.max_pages * a.c.page_size));
    const int blocks = (length + STEP - 1) / STEP, per = part_blocks(blocks, a.splits);
    const int first = split * per, last = min(blocks, first + per);
    if (first >= last && (a.splits > 1 || length > 0))
        return;                                                  // an empty part; the join does not read it

    // Pages of the lane's two granules of 8 tokens of a block, as a row of K
    // (col / 4) and as the holder of scores and values (g); -1: none.  Reads
    // stay inside the sequence's row of the table whatever the block.
    const int32_t *table = a.c.table + (int64_t)b * a.c.max_pages;
    const auto next_pages = [&](int block, int &pk, int &pg) {
        if constexpr (ONE) {
            pk = table[min(q4_page_of(a.c, block * STEP), a.c.max_pages - 1)];
        } else {
            pk = table[min(q4_page_of(a.c, block * STEP + 8 * (col / 4)), a.c.max_pages - 1)];
            pg = table[min(q4_page_of(a.c, block * STEP + 8 * g), a.c.max_pages - 1)];
        }
    };
    typedef AttentionBlock<D, GROUP> Block;
    // This lane's place in a block: as a row of K, and as holder of 8 tokens
    const int k_token = 8 * (col / 4) + (col & 3), g_token = 8 * g;
    const auto load = [&](int block, int pk, int pg, Block &x) {
        const int t0 = block * STEP;
        const uint32_t *kc, *kw, *vw, *vc;
        if constexpr (ONE) {
            const int page = __builtin_amdgcn_readfirstlane(pk);
            const bool there = page >= 0 && page < a.c.pages;
            const int64_t hp = (int64_t)(there ? page : 0) * a.c.heads + h;
            const int slot = t0 - q4_page_of(a.c, t0) * a.c.page_size;
            kc = a.c.k_codes + (hp * a.c.page_size + slot) * (D / 8) + k_token * (D / 8);
            kw = a.c.k_words + hp * GROUPS * a.c.page_size + slot + g_token;
            vw = a.c.v_words + hp * GROUPS * a.c.page_size + slot + g_token;
            vc = a.c.v_codes + (hp * (a.c.page_size / 8) + slot / 8) * D + (g * 16 + col) * BLOCKS;
            x.mine = there;
            x.whole = there && t0 + STEP <= length;
        } else {
            const int tk = t0 + 8 * (col / 4), tg = t0 + g_token;
            const bool there_k = tk < length && pk >= 0 && pk < a.c.pages;
            const bool there_g = tg < length && pg >= 0 && pg < a.c.pages;
            const int sk = tk - q4_page_of(a.c, tk) * a.c.page_size, sg = tg - q4_page_of(a.c, tg) * a.c.page_size;
            const int64_t hk = (int64_t)(there_k ? pk : 0) * a.c.heads + h, hg = (int64_t)(there_g ? pg : 0) * a.c.heads + h;
            kc = a.c.k_codes + (hk * a.c.page_size + sk + (col & 3)) * (D / 8);
            kw = a.c.k_words + hg * GROUPS * a.c.page_size + sg;
            vw = a.c.v_words + hg * GROUPS * a.c.page_size + sg;
            vc = a.c.v_codes + (hg * (a.c.page_size / 8) + sg / 8) * D + col * BLOCKS;
            x.mine = there_g;
            x.whole = __builtin_amdgcn_readfirstlane(__all(there_g && tg + 8 <= length));
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if constexpr (D == 64) {
                const uint2 v = *reinterpret_cast<const uint2 *>(kc + u * (4 * D / 8) + 2 * g);
                x.k[u][0] = v.x;
                x.k[u][1] = v.y;
            } else {
#pragma unroll
                for (int n = 0; n < D / 128; ++n) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(kc + u * (4 * D / 8) + 16 * n + 4 * g);
                    x.k[u][4 * n] = v.x;
                    x.k[u][4 * n + 1] = v.y;
                    x.k[u][4 * n + 2] = v.z;
                    x.k[u][4 * n + 3] = v.w;
                }
            }
        }
#pragma unroll
        for (int n = 0; n < GROUPS; ++n)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                x.k_words[u][n] = *reinterpret_cast<const uint4 *>(kw + n * a.c.page_size + 4 * u);
                x.v_words[u][n] = *reinterpret_cast<const uint4 *>(vw + n * a.c.page_size + 4 * u);
            }
#pragma unroll
        for (int i = 0; i < BLOCKS; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(vc + i);
            x.v[i] = v.x;
            x.v[i + 1] = v.y;
            x.v[i + 2] = v.z;
            x.v[i + 3] = v.w;
        }
    };

    // This lane's head of Q, elements 32 j + 8 g .. + 7; the sign of the scale
    // goes into it (exactly), so that the largest product is the largest score.
    half8 q[D / 32];
    const float scale = __builtin_fmaxf(__builtin_fabsf(a.scale) * kLog2e, 0x1p-126f);   // 0 would undo -infinity
    float q_sum[GROUPS];
    float4v start[GROUPS];         // takes the 64 off again
    const auto load_queries = [&]() {
        const half_t *row = a.Q + b * a.q_stride + (q_head + min(col, rows - 1)) * D + 8 * g;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            q[j] = *reinterpret_cast<const half8 *>(row + 32 * j);
            q[j] = a.scale < 0.0f ? -q[j] : q[j];
        }
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

    float base = -INFINITY, l = 0.0f;
    float4v acc[BLOCKS];
#pragma unroll
    for (int i = 0; i < BLOCKS; ++i)
        acc[i] = float4v{0, 0, 0, 0};

    const auto attend = [&](int block, const Block &y) {
        const int tg = block * STEP + g_token;
        // score / scale of tokens tg + 4 u + r
        float x[8];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int n = 0; n < GROUPS; ++n) {
                float4v s = start[n];
#pragma unroll
                for (int j = n * JG; j < (n + 1) * JG; ++j)
                    s = __builtin_amdgcn_mfma_f32_16x16x32_f16(q4_codes_64(y.k[u][j], bits), q[j], s, 0, 0, 0);
                const uint4 w = y.k_words[u][n];
                const unsigned word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float t = __builtin_fmaf(-(float)(word[r] >> 16), q_sum[n], s[r]);
                    x[4 * u + r] = n == 0 ? q4_scale(word[r]) * t : __builtin_fmaf(q4_scale(word[r]), t, x[4 * u + r]);
                }
            }
        unsigned word[GROUPS][8];
#pragma unroll
        for (int n = 0; n < GROUPS; ++n) {
            const uint4 w0 = y.v_words[0][n], w1 = y.v_words[1][n];
            const unsigned w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                word[n][i] = w[i];
        }
        if (!y.whole) {   // what lies behind the last token has no weight, whatever it is
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool there = y.mine && tg + i < length;
                x[i] = there ? x[i] : -INFINITY;
#pragma unroll
                for (int n = 0; n < GROUPS; ++n)
                    word[n][i] = there ? word[n][i] : 0u;
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
        most = column_max(most);
        top = column_max(top);
        // the place of the largest P', 0 for -infinity times 0 (no token, or scale 0)
        const float reach = __builtin_fmaf(most, scale, (float)__builtin_amdgcn_frexp_expf(top));
        const bool grown = reach > base + kTop;
        if (__any(grown)) {
            const float to = grown ? reach - kLift : base;
            const float fade = base == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(base - to);
            base = to;
            l *= fade;
#pragma unroll
            for (int i = 0; i < BLOCKS; ++i)
                acc[i] *= fade;
        }
        const float from = base == -INFINITY ? 0.0f : -base;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], scale, from));
            l += x[i];
        }
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
            const unsigned z0 = q4_zero(w[0] >> 16, w[1] >> 16).a, z1 = q4_zero(w[2] >> 16, w[3] >> 16).b,
                           z2 = q4_zero(w[4] >> 16, w[5] >> 16).a, z3 = q4_zero(w[6] >> 16, w[7] >> 16).b;
#pragma unroll
            for (int i = n * GROUP / 16; i < (n + 1) * GROUP / 16; ++i) {
                const half8 v = q4_codes(y.v[i], bits, z0, z1, z2, z3);
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, hi, acc[i], 0, 0, 0);
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, lo, acc[i], 0, 0, 0);
            }
        }
    };

    int block = first + wave, pk = 0, pg = 0;
    if (block < last) {
        next_pages(block, pk, pg);
        if constexpr (Block::REGISTERS <= 32) {
            // A block's loads go out before the one ahead of it is attended
            // to, its pages one block earlier still (and before that block's
            // loads: waiting for the pages must not wait for those).
            Block x0, x1;
            int pk1 = 0, pg1 = 0;
            next_pages(block + WAVES, pk1, pg1);
            load(block, pk, pg, x0);
            load_queries();
            for (;;) {
                if (block + WAVES >= last) {
                    attend(block, x0);
                    break;
                }
                next_pages(block + 2 * WAVES, pk, pg);
                load(block + WAVES, pk1, pg1, x1);
                attend(block, x0);
                block += WAVES;
                if (block + WAVES >= last) {
                    attend(block, x1);
                    break;
                }
                next_pages(block + 2 * WAVES, pk1, pg1);
                load(block + WAVES, pk, pg, x0);
                attend(block, x1);
                block += WAVES;
            }
        } else {
            // two blocks would not fit the registers; the other waves' work
            // covers the loads
            load_queries();
            for (; block < last; block += WAVES) {
                Block x;
                load(block, pk, pg, x);
                next_pages(block + WAVES, pk, pg);
                attend(block, x);
            }
        }
    }
    l = column_sum(l);

    // join the waves: lane (g, head) holds d = 16 i + 4 g + r of its head
#pragma unroll
    for (int i = 0; i < BLOCKS; ++i) {
        *reinterpret_cast<float4v *>(sums + (wave * 16 + col) * PITCH + 16 * i + 4 * g) = acc[i];
    }
    if (g == 0) {
        stats[wave * 32 + col] = base;
        stats[wave * 32 + 16 + col] = l;
    }
    __syncthreads();
    for (int e = tid; e < rows * (D / 4); e += 64 * WAVES) {
        const int row = e / (D / 4), d = e % (D / 4) * 4;
        float top = -INFINITY, total = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            top = __builtin_fmaxf(top, stats[w * 32 + row]);
        const float from = top == -INFINITY ? 0.0f : top;
        float4v v = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float f = __builtin_amdgcn_exp2f(stats[w * 32 + row] - from);
            total += f * stats[w * 32 + 16 + row];
            const float4v part = *reinterpret_cast<const float4v *>(sums + (w * 16 + row) * PITCH + d);
            v += f * part;
        }
        const int64_t head = (int64_t)b * a.q_heads + q_head + row;
        if (a.splits == 1) {
            store_quotient(a.out + head * D + d, v, total);
        } else {
            *reinterpret_cast<float4v *>(a.parts + (head * a.splits + split) * D + d) = v;
            if (d == 0) {
                float *ml = a.parts + (int64_t)a.c.batch * a.q_heads * a.splits * D + (head * a.splits + split) * 2;
                ml[0] = top;
                ml[1] = total;
            }
        }
    }
}

// Join the parts of the heads: D / 4 lanes hold a head's elements, and TEAMS
// teams of them take its parts in turn; the teams' sums are added in order.
// With one team a workgroup joins several heads.
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
        const int b = (int)(head / a.q_heads);
        const int length = (int)min((int64_t)max(a.lengths[b], 0), (int64_t)a.c.max_pages * a.c.page_size);
        const int blocks = (length + STEP - 1) / STEP, per = part_blocks(blocks, a.splits);
        const int used = per > 0 ? (blocks + per - 1) / per : 0;     // parts that hold tokens
        const float *ml = a.parts + heads * a.splits * D + head * a.splits * 2;
        const float *part = a.parts + head * a.splits * D + 4 * d;
        float top = -INFINITY;
        if constexpr (TEAMS > 1) {   // one head: every wave looks at all parts
            for (int s = threadIdx.x & 63; s < used; s += 64)
                top = __builtin_fmaxf(top, ml[2 * s]);
#pragma unroll
            for (int m = 1; m < 64; m *= 2)
                top = __builtin_fmaxf(top, __shfl_xor(top, m));
        } else {
#pragma unroll 4
            for (int s = 0; s < used; ++s)
                top = __builtin_fmaxf(top, ml[2 * s]);
        }
        const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll 4
        for (int s = team; s < used; s += TEAMS) {
            const float f = __builtin_amdgcn_exp2f(ml[2 * s] - base);
            total += f * ml[2 * s + 1];
            v += f * *reinterpret_cast<const float4v *>(part + (int64_t)s * D);
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

template <int D, int GROUP>
static hipError_t launch_attention(const Q4AttentionArgs &a, int64_t grid, hipStream_t s)
{
    if (a.c.page_size % STEP == 0)
        hipLaunchKernelGGL((q4_attention_kernel<D, GROUP, true>), dim3((unsigned)grid), dim3(64 * WAVES),
                           (unsigned)q4_attention_lds_bytes(D), s, a);
    else
        hipLaunchKernelGGL((q4_attention_kernel<D, GROUP, false>), dim3((unsigned)grid), dim3(64 * WAVES),
                           (unsigned)q4_attention_lds_bytes(D), s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1)
        return e;
    // few parts: a team for each head; many: all of a workgroup's teams
    const int64_t heads = (int64_t)a.c.batch * a.q_heads;
    constexpr int TEAMS = 1024 / D;
    if (a.splits <= 8)
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
