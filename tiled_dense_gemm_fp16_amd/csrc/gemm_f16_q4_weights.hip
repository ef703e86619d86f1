// gemm_f16_q4_weights.hip -- 4-bit weights: rounding a matrix to codes,
// reading it back, and the product C = epi(alpha A W^T) with it.
#include "gemm_f16_q4_format.h"
#include "gemm_f16_tile.h"

namespace gemm_f16_impl {

// ---- compress and expand ---------------------------------------------------------
// One wave per 16 x 128 tile.  Lane 16 g + n holds the tile's dwords of row n,
// k = 32 j + 8 g + 0..7: four 16-byte pieces of the row, and one 16-byte store
// of four dwords that is contiguous over the wave.  A group of 32 is one j of
// the four lanes g, 64 two of them, 128 all four.

template <int GROUP, bool VEC>
__global__ void __launch_bounds__(256) q4_compress_kernel(const half_t *__restrict__ W, uint32_t *__restrict__ codes,
                                                          uint32_t *__restrict__ words, int64_t N, int64_t K,
                                                          int64_t k_blocks, int64_t tiles, bool symmetric)
{
    constexpr int GROUPS = 128 / GROUP, PER = GROUP / 32;   // groups of a tile's row, j of a group
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const int64_t stride = (int64_t)gridDim.x * 4;
    for (int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); tile < tiles; tile += stride) {
        const int64_t row = tile / k_blocks * 16 + n, k0 = tile % k_blocks * 128 + 8 * g;
        float x[4][8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            half8 v = {};
            const int64_t k = k0 + 32 * j;
            if constexpr (VEC) {
                if (row < N && k < K)
                    v = *reinterpret_cast<const half8 *>(W + row * K + k);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (row < N && k + i < K)
                        v[i] = W[row * K + k + i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f = (float)v[i];
                x[j][i] = f == f ? f : 0.0f;
            }
        }
        uint32_t word[GROUPS];
        uint4 out;
        unsigned dw[4];
#pragma unroll
        for (int q = 0; q < GROUPS; ++q) {
            float lo = 0.0f, hi = 0.0f;
#pragma unroll
            for (int j = q * PER; j < (q + 1) * PER; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    lo = __builtin_fminf(lo, x[j][i]);
                    hi = __builtin_fmaxf(hi, x[j][i]);
                }
#pragma unroll
            for (int m = 16; m < 64; m *= 2) {
                lo = __builtin_fminf(lo, __shfl_xor(lo, m));
                hi = __builtin_fmaxf(hi, __shfl_xor(hi, m));
            }
            const q4_rounder r(lo, hi, symmetric);
            word[q] = r.word();
#pragma unroll
            for (int j = q * PER; j < (q + 1) * PER; ++j) {
                dw[j] = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    dw[j] |= r.code(x[j][i]) << q4_shift(i);
            }
        }
        out = make_uint4(dw[0], dw[1], dw[2], dw[3]);
        *reinterpret_cast<uint4 *>(codes + (tile * 64 + lane) * 4) = out;
        if (g == 0) {
#pragma unroll
            for (int q = 0; q < GROUPS; ++q)
                words[(tile * 16 + n) * GROUPS + q] = word[q];
        }
    }
}

template <int GROUP, bool VEC>
__global__ void __launch_bounds__(256) q4_expand_kernel(const uint32_t *__restrict__ codes,
                                                        const uint32_t *__restrict__ words, half_t *__restrict__ W,
                                                        int64_t N, int64_t K, int64_t k_blocks, int64_t tiles)
{
    constexpr int GROUPS = 128 / GROUP, PER = GROUP / 32;
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const int64_t stride = (int64_t)gridDim.x * 4;
    for (int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); tile < tiles; tile += stride) {
        const int64_t row = tile / k_blocks * 16 + n, k0 = tile % k_blocks * 128 + 8 * g;
        const uint4 c = *reinterpret_cast<const uint4 *>(codes + (tile * 64 + lane) * 4);
        const unsigned dw[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t word = words[(tile * 16 + n) * GROUPS + j / PER];
            const float s = q4_scale(word);
            const half8 q = q4_codes(dw[j], q4_zero(word));
            half8 v;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = (half_t)(s * (float)q[i]);
            const int64_t k = k0 + 32 * j;
            if constexpr (VEC) {
                if (row < N && k < K)
                    *reinterpret_cast<half8 *>(W + row * K + k) = v;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (row < N && k + i < K)
                        W[row * K + k + i] = v[i];
            }
        }
    }
}

template <bool VEC>
static hipError_t launch_compress(const _Float16 *W, uint32_t *codes, uint32_t *words, int64_t N, int64_t K, int group,
                                  bool symmetric, hipStream_t s)
{
    const int64_t kb = (K + 127) / 128, tiles = (N + 15) / 16 * kb;
    const dim3 grid((unsigned)std::min<int64_t>((tiles + 3) / 4, 256 * 32));
    if (group == 32)
        hipLaunchKernelGGL((q4_compress_kernel<32, VEC>), grid, dim3(256), 0, s, W, codes, words, N, K, kb, tiles, symmetric);
    else if (group == 64)
        hipLaunchKernelGGL((q4_compress_kernel<64, VEC>), grid, dim3(256), 0, s, W, codes, words, N, K, kb, tiles, symmetric);
    else
        hipLaunchKernelGGL((q4_compress_kernel<128, VEC>), grid, dim3(256), 0, s, W, codes, words, N, K, kb, tiles, symmetric);
    return hipGetLastError();
}

hipError_t launch_q4_compress(const _Float16 *W, uint32_t *codes, uint32_t *words, int64_t N, int64_t K, int group,
                              bool symmetric, bool vec, hipStream_t s)
{
    return vec ? launch_compress<true>(W, codes, words, N, K, group, symmetric, s)
               : launch_compress<false>(W, codes, words, N, K, group, symmetric, s);
}

template <bool VEC>
static hipError_t launch_expand(const uint32_t *codes, const uint32_t *words, _Float16 *W, int64_t N, int64_t K,
                                int group, hipStream_t s)
{
    const int64_t kb = (K + 127) / 128, tiles = (N + 15) / 16 * kb;
    const dim3 grid((unsigned)std::min<int64_t>((tiles + 3) / 4, 256 * 32));
    if (group == 32)
        hipLaunchKernelGGL((q4_expand_kernel<32, VEC>), grid, dim3(256), 0, s, codes, words, W, N, K, kb, tiles);
    else if (group == 64)
        hipLaunchKernelGGL((q4_expand_kernel<64, VEC>), grid, dim3(256), 0, s, codes, words, W, N, K, kb, tiles);
    else
        hipLaunchKernelGGL((q4_expand_kernel<128, VEC>), grid, dim3(256), 0, s, codes, words, W, N, K, kb, tiles);
    return hipGetLastError();
}

hipError_t launch_q4_expand(const uint32_t *codes, const uint32_t *words, _Float16 *W, int64_t N, int64_t K, int group,
                            bool vec, hipStream_t s)
{
    return vec ? launch_expand<true>(codes, words, W, N, K, group, s)
               : launch_expand<false>(codes, words, W, N, K, group, s);
}

// ---- product -----------------------------------------------------------------------
// A workgroup owns 16 MB rows of A and 16 NW rows of W; its waves take the
// 128-deep k blocks in turn and add up their sums at the end, in wave order.
// A wave's step is one load of a 1 KiB tile of codes (16 bytes a lane) for
// each 16 rows of W; codes become q - z in registers (exact in binary16) and
// go straight into v_mfma_f32_16x16x32_f16 as its second operand, so W never
// passes through LDS.  The first operand, A, is staged in LDS `chunk` k at a
// time.  Products of a group are summed in fp32 and enter the total times the
// group's scale, in fp32, so nothing is rounded before the end.  With W as
// the second operand a lane holds results of the W row whose codes it
// unpacked: zero point and scale are its own, with no exchange of lanes.

template <int GROUP, int MB, int NW, int WAVES>
__global__ void __launch_bounds__(64 * WAVES) q4_product_kernel(Q4Args p)
{
    constexpr int GROUPS = 128 / GROUP, PER = GROUP / 32;
    extern __shared__ __attribute__((aligned(16))) unsigned char q4_lds[];
    half_t *xs = reinterpret_cast<half_t *>(q4_lds);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int m0 = blockIdx.y * (16 * MB), nb0 = blockIdx.x * NW;
    const int rows = min(p.M - m0, 16 * MB), pitch = p.chunk + 8;

    float4v acc[MB][NW];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nw = 0; nw < NW; ++nw)
            acc[mb][nw] = float4v{0, 0, 0, 0};

    for (int c0 = 0; c0 < p.K; c0 += p.chunk) {
        // stage A's rows, k from c0, zeros past K (pitch: 16 bytes more than
        // the chunk, so that 16 rows' reads fall on different LDS banks)
        const int pieces = p.chunk / 8;
        for (int e = tid; e < rows * pieces; e += 64 * WAVES) {
            const int r = e / pieces, k = c0 + e % pieces * 8;
            const half_t *src = p.A + (int64_t)(m0 + r) * p.K + k;
            half8 v = {};
            if (p.vec_a) {
                if (k < p.K)
                    v = *reinterpret_cast<const half8 *>(src);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (k + i < p.K)
                        v[i] = src[i];
            }
            *reinterpret_cast<half8 *>(xs + r * pitch + (k - c0)) = v;
        }
        __syncthreads();
        const int end = min(p.k_blocks, (c0 + p.chunk) / 128);
        for (int kb = c0 / 128 + wave; kb < end; kb += WAVES) {
            unsigned dw[NW][4];
            unsigned word[NW][GROUPS];
#pragma unroll
            for (int nw = 0; nw < NW; ++nw) {
                const int64_t tile = (int64_t)min(nb0 + nw, p.n_blocks - 1) * p.k_blocks + kb;
                const uint4 c = *reinterpret_cast<const uint4 *>(p.codes + (tile * 64 + lane) * 4);
                dw[nw][0] = c.x;
                dw[nw][1] = c.y;
                dw[nw][2] = c.z;
                dw[nw][3] = c.w;
#pragma unroll
                for (int q = 0; q < GROUPS; ++q)
                    word[nw][q] = p.words[(tile * 16 + (lane & 15)) * GROUPS + q];
            }
            const half_t *x = xs + (kb * 128 - c0) + 8 * (lane >> 4);
#pragma unroll
            for (int q = 0; q < GROUPS; ++q) {
                float4v sum[MB][NW];
#pragma unroll
                for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                    for (int nw = 0; nw < NW; ++nw)
                        sum[mb][nw] = float4v{0, 0, 0, 0};
#pragma unroll
                for (int j = q * PER; j < (q + 1) * PER; ++j) {
                    half8 b[NW];
#pragma unroll
                    for (int nw = 0; nw < NW; ++nw)
                        b[nw] = q4_codes(dw[nw][j], q4_zero(word[nw][q]));
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb) {
                        const int r = min(16 * mb + (lane & 15), rows - 1);   // rows past M repeat the last one
                        const half8 a = *reinterpret_cast<const half8 *>(x + r * pitch + 32 * j);
#pragma unroll
                        for (int nw = 0; nw < NW; ++nw)
                            sum[mb][nw] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b[nw], sum[mb][nw], 0, 0, 0);
                    }
                }
#pragma unroll
                for (int nw = 0; nw < NW; ++nw) {
                    const float s = q4_scale(word[nw][q]);
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[mb][nw][r] += s * sum[mb][nw][r];
                }
            }
        }
        __syncthreads();
    }

    // add the waves' sums in wave order; lane (g, n) holds rows 4 g + r of
    // A, column n of each 16 x 16 block
    float4v *part = reinterpret_cast<float4v *>(q4_lds);   // [wave][mb][nw][lane]
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nw = 0; nw < NW; ++nw)
            part[((wave * MB + mb) * NW + nw) * 64 + lane] = acc[mb][nw];
    __syncthreads();
    const float *flat = reinterpret_cast<const float *>(part);
    for (int e = tid; e < rows * NW * 16; e += 64 * WAVES) {
        const int col = e % (NW * 16), m = e / (NW * 16);
        const int n = nb0 * 16 + col;
        if (n >= p.N)
            continue;
        const int at = (((m / 16) * NW + col / 16) * 64 + m % 16 / 4 * 16 + col % 16) * 4 + m % 4;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            v += flat[w * (MB * NW * 256) + at];
        v *= p.alpha;
        if (p.relu)
            v = __builtin_fmaxf(v, 0.0f);
        p.C[(int64_t)(m0 + m) * p.N + n] = (half_t)v;
    }
}

const Q4Config kQ4Configs[kNumQ4Configs] = {
    {"q4_16x16_w8", 1, 1, 8},
    {"q4_32x32_w8", 2, 2, 8},
    {"q4_64x32_w8", 4, 2, 8},
};

// k staged at a time: all of K when it fits in 64 KiB, and always a multiple
// of 128 k for each wave.
int q4_chunk(const Q4Config &c, int64_t M, int64_t K)
{
    const int64_t step = 128 * c.waves, rows = std::min<int64_t>(M, 16 * c.m_blocks);
    const int64_t fit = std::max<int64_t>(step, (65536 / (2 * rows) - 8) / step * step);
    return (int)std::min<int64_t>(fit, (K + step - 1) / step * step);
}

int64_t q4_lds_bytes(const Q4Config &c, int64_t M, int chunk)
{
    const int64_t rows = std::min<int64_t>(M, 16 * c.m_blocks);
    return std::max<int64_t>(rows * (chunk + 8) * 2, (int64_t)c.waves * c.m_blocks * c.n_blocks * 1024);
}

template <int GROUP>
static hipError_t launch_group(int config, const Q4Args &a, dim3 grid, unsigned lds, hipStream_t s)
{
    switch (config) {
    case 0: hipLaunchKernelGGL((q4_product_kernel<GROUP, 1, 1, 8>), grid, dim3(512), lds, s, a); break;
    case 1: hipLaunchKernelGGL((q4_product_kernel<GROUP, 2, 2, 8>), grid, dim3(512), lds, s, a); break;
    case 2: hipLaunchKernelGGL((q4_product_kernel<GROUP, 4, 2, 8>), grid, dim3(512), lds, s, a); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

hipError_t launch_q4(int config, int group, const Q4Args &a, int64_t grid_n, int64_t grid_m, hipStream_t s)
{
    const unsigned lds = (unsigned)q4_lds_bytes(kQ4Configs[config], a.M, a.chunk);
    // the second grid dimension is 16 bits: more rows go in several launches
    const int64_t step = 16 * kQ4Configs[config].m_blocks * (int64_t)65535;
    for (int64_t m = 0; m < a.M; m += step) {
        Q4Args b = a;
        b.A += m * a.K;
        b.C += m * a.N;
        b.M = (int)std::min<int64_t>(a.M - m, step);
        const dim3 grid((unsigned)grid_n, (unsigned)std::min<int64_t>(grid_m - m / step * 65535, 65535));
        const hipError_t e = group == 32   ? launch_group<32>(config, b, grid, lds, s)
                             : group == 64 ? launch_group<64>(config, b, grid, lds, s)
                                           : launch_group<128>(config, b, grid, lds, s);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

} // namespace gemm_f16_impl
