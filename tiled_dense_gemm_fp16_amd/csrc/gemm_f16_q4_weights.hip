// gemm_f16_q4_weights.hip -- 4-bit weights: rounding a matrix to codes,
// reading it back, and the product C = epi(alpha A W^T) with it.
#include "gemm_f16_q4_format.h"
#include "gemm_f16_tile.h"

namespace gemm_f16_impl {

// 16 bytes at any (2-byte) alignment: rows of an odd number of elements.  The
// memory path serves unaligned 16-byte accesses.
typedef _Float16 half8_any __attribute__((ext_vector_type(8), aligned(2)));

// Eight elements of a row of which `left` remain; zeros past its end.
__device__ __forceinline__ half8 row_piece(const half_t *p, int left)
{
    half8 v = {};
    if (left >= 8) {
        v = *reinterpret_cast<const half8_any *>(p);
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < left)
                v[i] = p[i];
    }
    return v;
}

// ---- rows made aligned ---------------------------------------------------------------
// 16 bytes a thread; the products over the copy are what this is for (bound by
// A's bytes, 3 us for 300 rows of 8193 with the launch).
__global__ void __launch_bounds__(256) q4_pack_kernel(const half_t *__restrict__ A, half_t *__restrict__ to, int64_t K,
                                                      int64_t chunks, int64_t pitch)
{
    const int64_t row = blockIdx.x / chunks;
    const int64_t k = (blockIdx.x % chunks * 256 + threadIdx.x) * 8;
    if (k < pitch)
        *reinterpret_cast<half8 *>(to + row * pitch + k) = row_piece(A + row * K + k, (int)(K - k < 8 ? K - k : 8));
}

hipError_t launch_q4_pack(const _Float16 *A, _Float16 *to, int64_t M, int64_t K, int64_t pitch, hipStream_t s)
{
    // workgroups of 2048 elements of a row; launches stay below 2^31 threads
    const int64_t chunks = (pitch + 2047) / 2048, rows = std::max<int64_t>(((int64_t)1 << 22) / chunks, 1);
    for (int64_t m = 0; m < M; m += rows)
        hipLaunchKernelGGL(q4_pack_kernel, dim3((unsigned)(std::min(rows, M - m) * chunks)), dim3(256), 0, s, A + m * K,
                           to + m * pitch, K, chunks, pitch);
    return hipGetLastError();
}

// ---- compress and expand ---------------------------------------------------------
// One wave per 16 x 128 tile.  Lane 16 g + n holds the tile's dwords of row n,
// k = 32 j + 8 g + 0..7: four 16-byte pieces of the row, and one 16-byte store
// of four dwords that is contiguous over the wave.  A group of 32 is one j of
// the four lanes g, 64 two of them, 128 all four.  Both kernels are bound by the
// matrix's bytes: at 8192 x 8192 compress takes 32 us (groups of 128; 34 with 32) and
// expand 32.5 (36), 5.3 and 5.2 TB/s, over inputs that no cache holds (26 to expand
// codes just written), and at 5000 x 4100 with groups of 32, whose rows are only
// 8-byte aligned, 15.5 and 16.6.  Compress reads the pieces as the tile has them, 64
// bytes of a row by four lanes (whole rows of 256 bytes at once, through LDS, took 35
// where this took 31); expand writes whole rows by way of LDS (64 bytes each took
// 38.5, where this took 32.7).

// A tile row's words, loaded and stored at once.
template <int GROUPS>
struct alignas(4 * GROUPS) q4_row_words {
    uint32_t w[GROUPS];
};

template <int GROUP>
__global__ void __launch_bounds__(256) q4_compress_kernel(const half_t *__restrict__ W, uint32_t *__restrict__ codes,
                                                          uint32_t *__restrict__ words, int64_t N, int64_t K,
                                                          int64_t k_blocks, int64_t tiles, bool symmetric)
{
    constexpr int GROUPS = 128 / GROUP, PER = GROUP / 32;   // groups of a tile's row, j of a group
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const int64_t stride = (int64_t)gridDim.x * 4;
    for (int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); tile < tiles; tile += stride) {
        const int64_t row = tile / k_blocks * 16 + n, k0 = tile % k_blocks * 128 + 8 * g;
        half8 x[4];
        half8 sum = {};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[j] = half8{};
            const int64_t k = k0 + 32 * j;
            if (row < N)
                x[j] = row_piece(W + row * K + k, (int)(K - k));
            sum += x[j];
        }
        // a NaN (or an infinity, or an overflow) shows in the sum: rare, so
        // the replacement of NaN is skipped without one
        bool odd = false;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            odd |= !(__builtin_fabsf((float)sum[i]) < 65504.0f);
        if (__any(odd)) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[j][i] = x[j][i] == x[j][i] ? x[j][i] : (half_t)0.0f;
        }
        q4_row_words<GROUPS> word;
        uint4 out;
        unsigned dw[4];
#pragma unroll
        for (int q = 0; q < GROUPS; ++q) {
            half8 low = x[q * PER], high = low;
#pragma unroll
            for (int j = q * PER + 1; j < (q + 1) * PER; ++j) {
                low = __builtin_elementwise_min(low, x[j]);
                high = __builtin_elementwise_max(high, x[j]);
            }
            float lo = 0.0f, hi = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                lo = __builtin_fminf(lo, (float)low[i]);
                hi = __builtin_fmaxf(hi, (float)high[i]);
            }
            q4_column_extremes(lo, hi);
            const q4_rounder r(lo, hi, symmetric);
            word.w[q] = r.word();
#pragma unroll
            for (int j = q * PER; j < (q + 1) * PER; ++j) {
                unsigned bits[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    bits[i] = r.code16((float)x[j][i]);
                dw[j] = r.join(bits);
            }
        }
        out = make_uint4(dw[0], dw[1], dw[2], dw[3]);
        *reinterpret_cast<uint4 *>(codes + (tile * 64 + lane) * 4) = out;
        if (g == 0)
            *reinterpret_cast<q4_row_words<GROUPS> *>(words + (tile * 16 + n) * GROUPS) = word;
    }
}

template <int GROUP>
__global__ void __launch_bounds__(256) q4_expand_kernel(const uint32_t *__restrict__ codes,
                                                        const uint32_t *__restrict__ words, half_t *__restrict__ W,
                                                        int64_t N, int64_t K, int64_t k_blocks, int64_t tiles)
{
    constexpr int GROUPS = 128 / GROUP, PER = GROUP / 32;
    const q4_bits bits;
    __shared__ half8 rows[4][16][17];   // [wave][row][piece]: 16 pieces, one more against bank conflicts
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    half8(&mine)[16][17] = rows[threadIdx.x >> 6];
    const int64_t stride = (int64_t)gridDim.x * 4;
    for (int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); tile < tiles; tile += stride) {
        const uint4 c = *reinterpret_cast<const uint4 *>(codes + (tile * 64 + lane) * 4);
        const unsigned dw[4] = {c.x, c.y, c.z, c.w};
        const q4_row_words<GROUPS> row_word = *reinterpret_cast<const q4_row_words<GROUPS> *>(words + (tile * 16 + n) * GROUPS);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t word = row_word.w[j / PER];
            const float s = q4_scale(word);
            const half8 q = q4_codes(dw[j], bits, q4_zero(word));
            half8 v;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = (half_t)(s * (float)q[i]);
            mine[n][4 * j + g] = v;
        }
        // whole rows of 256 bytes at once, as memory holds them
        q4_wave_fence();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = tile / k_blocks * 16 + 4 * i + g, k = tile % k_blocks * 128 + 8 * n;
            const half8 v = mine[4 * i + g][n];
            if (row < N && k + 8 <= K) {
                *reinterpret_cast<half8_any *>(W + row * K + k) = v;
            } else if (row < N) {
#pragma unroll
                for (int e = 0; e < 7; ++e)
                    if (k + e < K)
                        W[row * K + k + e] = v[e];
            }
        }
        q4_wave_fence();
    }
}

template <int GROUP>
static void launch_compress(const _Float16 *W, uint32_t *codes, uint32_t *words, int64_t N, int64_t K, bool symmetric,
                            hipStream_t s)
{
    const int64_t kb = (K + 127) / 128, tiles = (N + 15) / 16 * kb;
    const dim3 grid((unsigned)std::min<int64_t>((tiles + 3) / 4, 256 * 32));
    hipLaunchKernelGGL((q4_compress_kernel<GROUP>), grid, dim3(256), 0, s, W, codes, words, N, K, kb, tiles, symmetric);
}

hipError_t launch_q4_compress(const _Float16 *W, uint32_t *codes, uint32_t *words, int64_t N, int64_t K, int group,
                              bool symmetric, hipStream_t s)
{
    (group == 32 ? launch_compress<32> : group == 64 ? launch_compress<64> : launch_compress<128>)(W, codes, words, N, K,
                                                                                                 symmetric, s);
    return hipGetLastError();
}

template <int GROUP>
static void launch_expand(const uint32_t *codes, const uint32_t *words, _Float16 *W, int64_t N, int64_t K, hipStream_t s)
{
    const int64_t kb = (K + 127) / 128, tiles = (N + 15) / 16 * kb;
    const dim3 grid((unsigned)std::min<int64_t>((tiles + 3) / 4, 256 * 32));
    hipLaunchKernelGGL((q4_expand_kernel<GROUP>), grid, dim3(256), 0, s, codes, words, W, N, K, kb, tiles);
}

hipError_t launch_q4_expand(const uint32_t *codes, const uint32_t *words, _Float16 *W, int64_t N, int64_t K, int group,
                            hipStream_t s)
{
    (group == 32 ? launch_expand<32> : group == 64 ? launch_expand<64> : launch_expand<128>)(codes, words, W, N, K, s);
    return hipGetLastError();
}

// ---- product, few rows ---------------------------------------------------------------
// A workgroup owns 16 MB rows of A and 16 NW rows of W; its waves take the
// 128-deep k blocks in turn and add up their sums at the end, in wave order.
// A wave's step is one load of a 1 KiB tile of codes (16 bytes a lane) for
// each 16 rows of W; codes become q - z in registers (exact in binary16) and
// go straight into v_mfma_f32_16x16x32_f16 as its second operand.  The first
// operand, A, comes straight from memory in the layout of the instruction
// (lane (g, m) takes 16 bytes at k = 32 j + 8 g of row m): the waves split K,
// so no element of A is needed by two waves and LDS would only add a barrier.
// Products of a group are summed in fp32 and enter the total times the
// group's scale, in fp32, so nothing is rounded before the end.  With W as
// the second operand a lane holds results of the W row whose codes it
// unpacked: zero point and scale are its own, with no exchange of lanes.
//
// DEPTH steps are in flight: the kernel is bound by the latency and bandwidth
// of the codes' loads.  They are buffer loads, so that steps past the end,
// rows past M and rows of W past N read nothing (and return zeros) without a
// branch, which would make the compiler wait for more than it needs.  A whose
// rows are only 2-byte aligned is read by plain loads instead (ALIGNED false).
//
// 1 x 28672 x 8192 with groups of 128 takes 26.2 us, 4.8 TB/s of codes and words,
// 0.92 of what a copy reaches; 13 x 5000 x 4100 with groups of 32, one round of
// workgroups of which each wave takes 4 or 5 blocks one after the other, 7.6 us.  A wider
// workgroup of 64 x 128 outputs spills (43 us at 64 x 8192 x 8192, 27 with 4 waves).

template <int GROUPS>
__device__ __forceinline__ void load_words(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t at, unsigned (&w)[GROUPS])
{
    if constexpr (GROUPS == 1) {
        w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, off, at, 0);
    } else if constexpr (GROUPS == 2) {
        const auto v = __builtin_amdgcn_raw_buffer_load_b64(r, off, at, 0);
        w[0] = v[0];
        w[1] = v[1];
    } else {
        const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, off, at, 0);
        w[0] = v[0];
        w[1] = v[1];
        w[2] = v[2];
        w[3] = v[3];
    }
}

template <int GROUPS, int MB, int NW>
struct ProductStep {
    unsigned codes[NW][4];
    unsigned words[NW][GROUPS];
    half8 x[MB][4];
};

template <int GROUP, int MB, int NW, int WAVES, int DEPTH, bool ALIGNED>
__global__ void __launch_bounds__(64 * WAVES) q4_product_kernel(Q4Args p)
{
    constexpr int GROUPS = 128 / GROUP, PER = GROUP / 32;
    extern __shared__ __attribute__((aligned(16))) unsigned char q4_lds[];
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m0 = blockIdx.y * (16 * MB), nb0 = blockIdx.x * NW;
    const int rows = min(p.M - m0, 16 * MB), here = min(NW, p.n_blocks - nb0);
    const q4_bits bits;

    const __amdgpu_buffer_rsrc_t codes = make_rsrc(p.codes + (int64_t)nb0 * p.k_blocks * 256,
                                                   (uint32_t)here * (uint32_t)p.k_blocks * 1024u);
    const __amdgpu_buffer_rsrc_t words = make_rsrc(p.words + (int64_t)nb0 * p.k_blocks * (16 * GROUPS),
                                                   (uint32_t)here * (uint32_t)p.k_blocks * (64u * GROUPS));
    const __amdgpu_buffer_rsrc_t a = make_rsrc(p.A + (int64_t)m0 * p.K, (uint32_t)rows * (uint32_t)p.K * 2u);
    const half_t *row[MB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
        row[mb] = p.A + (int64_t)(m0 + min(16 * mb + col, rows - 1)) * p.K + 8 * g;

    typedef ProductStep<GROUPS, MB, NW> Step;
    const auto load_w = [&](int kb, uint32_t gone, Step &s, int from, int to) {
#pragma unroll
        for (int nw = from; nw < to; ++nw) {
            const uint32_t tile = (uint32_t)nw * (uint32_t)p.k_blocks;
            const auto v = __builtin_amdgcn_raw_buffer_load_b128(codes, (tile * 1024u + lane * 16u) | gone,
                                                                 (uint32_t)kb * 1024u, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s.codes[nw][i] = v[i];
            load_words<GROUPS>(words, (tile * (64u * GROUPS) + col * (4u * GROUPS)) | gone, (uint32_t)kb * (64u * GROUPS),
                               s.words[nw]);
        }
    };
    // this split's k blocks, and those of them that A's rows fill
    const int begin = blockIdx.z * p.split_blocks, end = min(p.k_blocks, begin + p.split_blocks);
    const int whole = min(p.K / 128, end);
    const auto load_x = [&](int kb, Step &s) {
        const uint32_t gone = oob_unless(kb < whole);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (ALIGNED) {
                    const uint32_t off = (uint32_t)(16 * mb + col) * (uint32_t)p.K * 2u + 16u * g + 64u * j;
                    s.x[mb][j] = __builtin_bit_cast(
                        half8, __builtin_amdgcn_raw_buffer_load_b128(a, off | gone, (uint32_t)kb * 256u, 0));
                } else {
                    s.x[mb][j] = *reinterpret_cast<const half8_any *>(row[mb] + max(0, min(kb, whole - 1)) * 128 + 32 * j);
                }
            }
    };

    float4v acc[MB][NW];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nw = 0; nw < NW; ++nw)
            acc[mb][nw] = float4v{0, 0, 0, 0};

    const auto load = [&](int kb, Step &s) {
        load_w(kb, oob_unless(kb < whole), s, 0, NW);
        load_x(kb, s);
    };
    const auto multiply = [&](const Step &s, int from, int to) {
#pragma unroll
        for (int nw = from; nw < to; ++nw) {
#pragma unroll
            for (int q = 0; q < GROUPS; ++q) {
                const q4_zero zero(s.words[nw][q]);
                const float scale = q4_scale(s.words[nw][q]);
                float4v sum[MB];
#pragma unroll
                for (int j = q * PER; j < (q + 1) * PER; ++j) {
                    const half8 w = q4_codes(s.codes[nw][j], bits, zero);
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb)
                        sum[mb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                            s.x[mb][j], w, j == q * PER ? float4v{0, 0, 0, 0} : sum[mb], 0, 0, 0);
                }
#pragma unroll
                for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[mb][nw][r] = __builtin_fmaf(scale, sum[mb][r], acc[mb][nw][r]);
            }
        }
    };

    const int first = begin + wave;
    if (first < whole) {
        if constexpr (DEPTH == 1) {
            // one step's registers: each part is loaded again for the next
            // step as soon as it has been used
            Step s;
            load(first, s);
            for (int kb = first; kb < whole; kb += WAVES) {
                const int next = kb + WAVES;
#pragma unroll
                for (int nw = 0; nw < NW; ++nw) {
                    multiply(s, nw, nw + 1);
                    load_w(next, oob_unless(next < whole), s, nw, nw + 1);
                }
                load_x(next, s);
            }
        } else {
            Step s[DEPTH];
#pragma unroll
            for (int d = 0; d < DEPTH; ++d)
                load(first + d * WAVES, s[d]);
            for (int kb = first;; kb += DEPTH * WAVES) {
                bool done = false;
#pragma unroll
                for (int d = 0; d < DEPTH; ++d) {
                    multiply(s[d], 0, NW);
                    if (kb + (d + 1) * WAVES >= whole) {
                        done = true;
                        break;
                    }
                    load(kb + (d + DEPTH) * WAVES, s[d]);
                }
                if (done)
                    break;
            }
        }
    }
    if (whole < end && wave == (whole - begin) % WAVES) {   // the k block that A's rows end in
        Step s;
        load_w(whole, 0u, s, 0, NW);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s.x[mb][j] = row_piece(row[mb] + whole * 128 + 32 * j, p.K - whole * 128 - 8 * g - 32 * j);
        multiply(s, 0, NW);
    }

    // add the waves' sums in wave order, CHUNK of the 16-column blocks at a
    // time; lane (g, col) holds rows 4 g + r of A, column col of each block
    constexpr int CHUNK = q4_sum_chunk(MB, NW);
    float4v *part = reinterpret_cast<float4v *>(q4_lds);   // [wave][mb][nw of the chunk][lane]
    const float *flat = reinterpret_cast<const float *>(q4_lds);
#pragma unroll
    for (int c = 0; c < NW; c += CHUNK) {
        if (c > 0)
            __syncthreads();
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int nw = 0; nw < CHUNK; ++nw)
                part[((wave * MB + mb) * CHUNK + nw) * 64 + lane] = acc[mb][c + nw];
        __syncthreads();
        for (int e = tid; e < rows * CHUNK * 16; e += 64 * WAVES) {
            const int at_n = e % (CHUNK * 16), m = e / (CHUNK * 16);
            const int n = (nb0 + c) * 16 + at_n;
            if (n >= p.N)
                continue;
            const int at = (((m / 16) * CHUNK + at_n / 16) * 64 + m % 16 / 4 * 16 + at_n % 16) * 4 + m % 4;
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w)
                v += flat[w * (MB * CHUNK * 256) + at];
            if (p.W) {   // a split's partial sums, joined by the reduction kernel
                p.W[((int64_t)blockIdx.z * p.rows + p.row0 + m0 + m) * p.N + n] = v;
                continue;
            }
            v *= p.alpha;
            if (p.relu)
                v = __builtin_fmaxf(v, 0.0f);
            p.C[(int64_t)(m0 + m) * p.N + n] = (half_t)v;
        }
    }
}

template <int GROUP, bool ALIGNED>
static hipError_t launch_group(int config, const Q4Args &a, dim3 grid, unsigned lds, hipStream_t s)
{
    // steps in flight: no more than the waves have
    const bool one = a.split_blocks <= 8;
    switch (config) {
    case 0:
        if (one)
            hipLaunchKernelGGL((q4_product_kernel<GROUP, 1, 1, 8, 1, ALIGNED>), grid, dim3(512), lds, s, a);
        else
            hipLaunchKernelGGL((q4_product_kernel<GROUP, 1, 1, 8, 4, ALIGNED>), grid, dim3(512), lds, s, a);
        break;
    case 1:
        if (one)
            hipLaunchKernelGGL((q4_product_kernel<GROUP, 1, 2, 8, 1, ALIGNED>), grid, dim3(512), lds, s, a);
        else
            hipLaunchKernelGGL((q4_product_kernel<GROUP, 1, 2, 8, 3, ALIGNED>), grid, dim3(512), lds, s, a);
        break;
    case 2: hipLaunchKernelGGL((q4_product_kernel<GROUP, 1, 4, 8, 2, ALIGNED>), grid, dim3(512), lds, s, a); break;
    case 3: hipLaunchKernelGGL((q4_product_kernel<GROUP, 2, 4, 8, 1, ALIGNED>), grid, dim3(512), lds, s, a); break;
    case 4: hipLaunchKernelGGL((q4_product_kernel<GROUP, 2, 8, 8, 1, ALIGNED>), grid, dim3(512), lds, s, a); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <int GROUP>
static hipError_t launch_aligned(int config, const Q4Args &a, dim3 grid, unsigned lds, hipStream_t s)
{
    return (uintptr_t)a.A % 4 == 0 && a.K % 2 == 0 ? launch_group<GROUP, true>(config, a, grid, lds, s)
                                                   : launch_group<GROUP, false>(config, a, grid, lds, s);
}

hipError_t launch_q4(int config, int group, const Q4Args &a, hipStream_t s)
{
    const unsigned lds = (unsigned)q4_lds_bytes(kQ4Configs[config], group);
    // the second grid dimension is 16 bits: more rows go in several launches
    const int64_t step = 16 * kQ4Configs[config].m_blocks * (int64_t)65535;
    for (int64_t m = 0; m < a.M; m += step) {
        Q4Args b = a;
        b.A += m * a.K;
        b.C += m * a.N;
        b.row0 = (int)m;
        b.M = (int)std::min<int64_t>(a.M - m, step);
        const dim3 grid((unsigned)a.tiles_n, (unsigned)std::min<int64_t>(a.tiles_m - m / step * 65535, 65535),
                        (unsigned)a.splits);
        const hipError_t e = group == 32   ? launch_aligned<32>(config, b, grid, lds, s)
                             : group == 64 ? launch_aligned<64>(config, b, grid, lds, s)
                                           : launch_aligned<128>(config, b, grid, lds, s);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

} // namespace gemm_f16_impl
