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
// Codes enter as q (exact); with a group's scale s and zero point z the score
// is the sum over groups of s (q . x - z (sum of the group's x)), in fp32.
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
// exact.  P' enters as two binary16 parts (22 bits), so that the output
// carries no error beyond fp32's and its own rounding.  P' is held relative to
// 2^E >= the largest scale seen (E: running, per group of d) and times 2^14,
// so that neither small scales nor small probabilities leave binary16's range.
#include "gemm_f16_q4_format.h"
#include "gemm_f16_tile.h"

namespace gemm_f16_impl {

constexpr int WAVES = kQ4AttentionWaves, STEP = kQ4AttentionTokens;
constexpr float kLog2e = 1.4426950408889634f;

// Two values rounded towards zero to binary16, packed.  Only for splitting a
// value into two parts: the second takes up what the first leaves.
__device__ __forceinline__ q4_half2 pack_rtz(float a, float b)
{
    return __builtin_bit_cast(q4_half2, __builtin_amdgcn_cvt_pkrtz(a, b));
}

// q - z of a dword that holds one d of 8 tokens with zero points z[0..7].
struct token_zeros {
    unsigned a01, b23, a45, b67;
};
__device__ __forceinline__ half8 token_codes(unsigned w, const token_zeros &z)
{
    const q4_half2 p0 = q4_pair((w & 0x000F000Fu) | 0x64006400u, z.a01);
    const q4_half2 p1 = q4_pair((w & 0x00F000F0u) | 0x54005400u, z.b23);
    w >>= 8;
    const q4_half2 p2 = q4_pair((w & 0x000F000Fu) | 0x64006400u, z.a45);
    const q4_half2 p3 = q4_pair((w & 0x00F000F0u) | 0x54005400u, z.b67);
    return half8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

template <int D, int GROUP>
__global__ void __launch_bounds__(64 * WAVES) q4_attention_kernel(Q4AttentionArgs a)
{
    constexpr int GROUPS = D / GROUP, JG = GROUP / 32, BLOCKS = D / 16, PITCH = D + 4;
    extern __shared__ __attribute__((aligned(16))) unsigned char q4_attention_lds[];
    float *sums = reinterpret_cast<float *>(q4_attention_lds);   // [wave][16 heads][PITCH]
    float *stats = sums + WAVES * 16 * PITCH;                    // [wave][m, l][16 heads]

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, g = lane >> 4;
    int id = blockIdx.x;
    const int split = id % a.splits;
    id /= a.splits;
    const int tile = id % a.row_tiles;
    id /= a.row_tiles;
    const int h = id % a.c.heads, b = id / a.c.heads;
    const int rows = min(a.ratio - 16 * tile, 16);               // query heads of this workgroup
    const int64_t q_head = (int64_t)h * a.ratio + 16 * tile;

    const int64_t room = (int64_t)a.c.max_pages * a.c.page_size;
    const int length = (int)min((int64_t)max(a.lengths[b], 0), room);
    const int blocks = (length + STEP - 1) / STEP, per = (blocks + a.splits - 1) / a.splits;
    const int first = split * per, last = min(blocks, first + per);
    if (first >= last && (a.splits > 1 || length > 0))
        return;                                                  // an empty part; the join does not read it

    // this lane's head of Q, elements 32 j + 8 g .. + 7
    half8 q[D / 32];
    float q_sum[GROUPS];
    {
        const half_t *row = a.Q + b * a.q_stride + (q_head + min(col, rows - 1)) * D + 8 * g;
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
            q[j] = *reinterpret_cast<const half8 *>(row + 32 * j);
#pragma unroll
        for (int n = 0; n < GROUPS; ++n) {
            float t = 0.0f;
#pragma unroll
            for (int j = n * JG; j < (n + 1) * JG; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    t += (float)q[j][i];
            t += __shfl_xor(t, 16);
            q_sum[n] = t + __shfl_xor(t, 32);
        }
    }
    const float scale = a.scale * kLog2e;
    const q4_zero no_zero(0u);

    float m = -INFINITY, l = 0.0f;
    float4v acc[BLOCKS];
    int E[GROUPS];
#pragma unroll
    for (int i = 0; i < BLOCKS; ++i)
        acc[i] = float4v{0, 0, 0, 0};
#pragma unroll
    for (int n = 0; n < GROUPS; ++n)
        E[n] = -100;

    for (int block = first + wave; block < last; block += WAVES) {
        const int t0 = block * STEP;
        // page of the lane's two granules of 8 tokens: as a row of K (col / 4)
        // and as the holder of scores and values (g)
        const int tk = t0 + 8 * (col / 4), tg = t0 + 8 * g;
        const int pk = q4_page(a.c, b, tk), pg = q4_page(a.c, b, tg);
        const int sk = tk % a.c.page_size, sg = tg % a.c.page_size;
        const int64_t hk = (int64_t)max(pk, 0) * a.c.heads + h, hg = (int64_t)max(pg, 0) * a.c.heads + h;
        const bool whole = __all(pg >= 0 && tg + 8 <= length);

        // scores of tokens tg + 4 u + r
        float x[8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t *codes = a.c.k_codes + (hk * a.c.page_size + sk + 4 * u + (col & 3)) * (D / 8);
            unsigned dw[D / 32];
            if constexpr (D == 64) {
                const uint2 v = *reinterpret_cast<const uint2 *>(codes + 2 * g);
                dw[0] = v.x;
                dw[1] = v.y;
            } else {
#pragma unroll
                for (int n = 0; n < D / 128; ++n) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(codes + 16 * n + 4 * g);
                    dw[4 * n] = v.x;
                    dw[4 * n + 1] = v.y;
                    dw[4 * n + 2] = v.z;
                    dw[4 * n + 3] = v.w;
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
                x[4 * u + r] = 0.0f;
#pragma unroll
            for (int n = 0; n < GROUPS; ++n) {
                float4v s = {0, 0, 0, 0};
#pragma unroll
                for (int j = n * JG; j < (n + 1) * JG; ++j)
                    s = __builtin_amdgcn_mfma_f32_16x16x32_f16(q4_codes(dw[j], no_zero), q[j], s, 0, 0, 0);
                const uint4 w = *reinterpret_cast<const uint4 *>(a.c.k_words + (hg * GROUPS + n) * a.c.page_size + sg + 4 * u);
                const unsigned word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    x[4 * u + r] += q4_scale(word[r]) * (s[r] - (float)(word[r] >> 16) * q_sum[n]);
            }
        }
        float most = -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = whole || (pg >= 0 && tg + i < length) ? x[i] * scale : -INFINITY;
            most = __builtin_fmaxf(most, x[i]);
        }
        most = __builtin_fmaxf(most, __shfl_xor(most, 16));
        most = __builtin_fmaxf(most, __shfl_xor(most, 32));
        const float m_new = __builtin_fmaxf(m, most), base = m_new == -INFINITY ? 0.0f : m_new;
        const float fade = __builtin_amdgcn_exp2f(m - base);   // 0 for the first tokens
        m = m_new;
        l *= fade;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = __builtin_amdgcn_exp2f(x[i] - base);
            l += x[i];
        }

#pragma unroll
        for (int n = 0; n < GROUPS; ++n) {
            const uint4 *words = reinterpret_cast<const uint4 *>(a.c.v_words + (hg * GROUPS + n) * a.c.page_size + sg);
            const uint4 w0 = words[0], w1 = words[1];
            unsigned word[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
            if (!whole) {   // whatever lies behind the last token counts as zeros
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    word[i] = pg >= 0 && tg + i < length ? word[i] : 0u;
            }
            float s[8], top = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[i] = q4_scale(word[i]);
                top = __builtin_fmaxf(top, __builtin_fabsf(s[i]));
            }
            top = __builtin_fmaxf(top, __shfl_xor(top, 16));
            top = __builtin_fmaxf(top, __shfl_xor(top, 32));
            const int e = max(E[n], top > 0.0f ? __builtin_amdgcn_frexp_expf(top) : -100);
            const float shrink = fade * __builtin_amdgcn_ldexpf(1.0f, E[n] - e);
            E[n] = e;
            const float lift = __builtin_amdgcn_ldexpf(1.0f, 14 - e);
            half8 hi, lo;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float p0 = x[i] * (s[i] * lift), p1 = x[i + 1] * (s[i + 1] * lift);
                const q4_half2 v = pack_rtz(p0, p1), rest = pack_rtz(p0 - (float)v[0], p1 - (float)v[1]);
                hi[i] = v[0];
                hi[i + 1] = v[1];
                lo[i] = rest[0];
                lo[i + 1] = rest[1];
            }
            const token_zeros zeros = {q4_zero(word[0] >> 16, word[1] >> 16).a, q4_zero(word[2] >> 16, word[3] >> 16).b,
                                       q4_zero(word[4] >> 16, word[5] >> 16).a, q4_zero(word[6] >> 16, word[7] >> 16).b};
            const uint32_t *codes = a.c.v_codes + ((hg * (a.c.page_size / 8) + sg / 8) * 16 + col) * BLOCKS;
#pragma unroll
            for (int i = n * GROUP / 16; i < (n + 1) * GROUP / 16; ++i) {
                const half8 v = token_codes(codes[i], zeros);
                acc[i] *= shrink;
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, hi, acc[i], 0, 0, 0);
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, lo, acc[i], 0, 0, 0);
            }
        }
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);

    // join the waves: lane (g, head) holds d = 16 i + 4 g + r of its head
#pragma unroll
    for (int i = 0; i < BLOCKS; ++i) {
        const float unit = __builtin_amdgcn_ldexpf(1.0f, E[i * 16 / GROUP] - 14);
        float4v v = acc[i];
        v *= unit;
        *reinterpret_cast<float4v *>(sums + (wave * 16 + col) * PITCH + 16 * i + 4 * g) = v;
    }
    if (g == 0) {
        stats[wave * 32 + col] = m;
        stats[wave * 32 + 16 + col] = l;
    }
    __syncthreads();
    for (int e = tid; e < rows * (D / 4); e += 64 * WAVES) {
        const int row = e / (D / 4), d = e % (D / 4) * 4;
        float top = -INFINITY, total = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            top = __builtin_fmaxf(top, stats[w * 32 + row]);
        const float base = top == -INFINITY ? 0.0f : top;
        float4v v = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float f = __builtin_amdgcn_exp2f(stats[w * 32 + row] - base);
            total += f * stats[w * 32 + 16 + row];
            const float4v part = *reinterpret_cast<const float4v *>(sums + (w * 16 + row) * PITCH + d);
            v += f * part;
        }
        const int64_t head = (int64_t)b * a.q_heads + q_head + row;
        if (a.splits == 1) {
            const float inv = total > 0.0f ? 1.0f / total : total == 0.0f ? 0.0f : total;   // no tokens: zeros; NaN stays
            half4 out;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                out[r] = (half_t)(v[r] * inv);
            *reinterpret_cast<half4 *>(a.out + head * D + d) = out;
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

// Join the parts of each head in order: D / 4 lanes a head.
template <int D>
__global__ void __launch_bounds__(256) q4_attention_join_kernel(Q4AttentionArgs a)
{
    constexpr int LANES = D / 4;
    const int64_t head = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
    if (head >= (int64_t)a.c.batch * a.q_heads)
        return;
    const int d = threadIdx.x % LANES * 4, b = (int)(head / a.q_heads);
    const int64_t room = (int64_t)a.c.max_pages * a.c.page_size;
    const int length = (int)min((int64_t)max(a.lengths[b], 0), room);
    const int blocks = (length + STEP - 1) / STEP, per = (blocks + a.splits - 1) / a.splits;
    const int used = per > 0 ? (blocks + per - 1) / per : 0;     // parts that hold tokens
    const float *ml = a.parts + (int64_t)a.c.batch * a.q_heads * a.splits * D + head * a.splits * 2;
    const float *part = a.parts + head * a.splits * D + d;
    float top = -INFINITY;
    for (int s = 0; s < used; ++s)
        top = __builtin_fmaxf(top, ml[2 * s]);
    const float base = top == -INFINITY ? 0.0f : top;
    float total = 0.0f;
    float4v v = {0, 0, 0, 0};
    for (int s = 0; s < used; ++s) {
        const float f = __builtin_amdgcn_exp2f(ml[2 * s] - base);
        total += f * ml[2 * s + 1];
        v += f * *reinterpret_cast<const float4v *>(part + (int64_t)s * D);
    }
    const float inv = total > 0.0f ? 1.0f / total : total == 0.0f ? 0.0f : total;
    half4 out;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        out[r] = (half_t)(v[r] * inv);
    *reinterpret_cast<half4 *>(a.out + head * D + d) = out;
}

int64_t q4_attention_lds_bytes(int head_dim) { return 4 * WAVES * (16 * (head_dim + 4) + 32); }

template <int D, int GROUP>
static hipError_t launch_attention(const Q4AttentionArgs &a, int64_t grid, hipStream_t s)
{
    hipLaunchKernelGGL((q4_attention_kernel<D, GROUP>), dim3((unsigned)grid), dim3(64 * WAVES),
                       (unsigned)q4_attention_lds_bytes(D), s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1)
        return e;
    const int64_t heads = (int64_t)a.c.batch * a.q_heads, per = 256 / (D / 4);
    hipLaunchKernelGGL((q4_attention_join_kernel<D>), dim3((unsigned)((heads + per - 1) / per)), dim3(256), 0, s, a);
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
