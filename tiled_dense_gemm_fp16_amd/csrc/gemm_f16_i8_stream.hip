// gemm_f16_i8_stream.hip -- the product of few rows with 8-bit weights: each
// weight is read once, straight from memory into the matrix instruction.
//
// A workgroup owns 16 rows of A (of one expert's pairs) and 16 rows of W; its
// waves split K in steps of 256.  Lane (g, i) of v_mfma_i32_16x16x64_i8 takes 16
// codes of row i of an operand, k = 16 g .. 16 g + 15 of the step's 64, which is how
// rows lie in memory: a load of 16 bytes a lane feeds it with nothing in between,
// and no code is needed by two waves, so LDS would only add a barrier.  W is the
// first operand, so a lane holds four neighbouring columns of one row of C.  The
// waves' sums are integers; they are added through LDS at the end.
//
// Loads are buffer loads: rows past the last, and chunks past K (whole 16-byte
// chunks: K is a multiple of 16 here), read zeros without a branch.
//
// Bound by memory: 1 x 28672 x 8192 41 to 44 us, 5.3 to 5.7 TB/s; by the launch where W
// is small: 1 x 1024 x 1024 3.3 us.
#include "gemm_f16_i8_device.h"

namespace gemm_f16_impl {

namespace {

constexpr int kWaves = 8;
constexpr int kChunks = kI8StreamK / 64;   // matrix instructions of a step for each 16 rows of W

// (As written it takes 55 registers, which leaves room for four workgroups on a CU; over
// experts 79, for three.
// Forms that take 83, for two workgroups, need 48 us for 1 x 28672 x 8192, with one
// step at a time 43 to 45.)
constexpr int NB = 1;      // blocks of 16 rows of W for a workgroup: 2 and 4 take 53 and 57 us there
constexpr int DEPTH = 2;   // steps of a wave asked for ahead

template <bool EXPERTS>
__global__ void __launch_bounds__(64 * kWaves) i8_stream_kernel(I8Args p)
{
    __shared__ __attribute__((aligned(16))) int4v part[kWaves][NB][64];
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, i = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    I8Tile t;
    const int8_t *W = p.W;
    const float *w_scales = p.w_scales;
    int pair, row;   // of lane i's row of A; -1: none
    if constexpr (EXPERTS) {
        bool quarter;
        if (!i8_find_tile<16, 16 * NB, false>(p, blockIdx.x, lane, t, quarter))
            return;
        pair = i8_pair(p, t, i);
        row = pair < 0 ? -1 : pair / p.pairs_per_row;
        W += (int64_t)t.expert * p.N * p.w_pitch;
        w_scales += (int64_t)t.expert * p.N;
    } else {
        t.n0 = blockIdx.x % p.tiles_n * (16 * NB);
        t.first = blockIdx.x / p.tiles_n % p.tiles_m * 16;
        t.rows = min(16, p.M - t.first);
        row = i < t.rows ? t.first + i : -1;
        pair = row;
    }
    const int n0 = t.n0;
    const int split = EXPERTS ? 0 : blockIdx.x / p.tiles_n / p.tiles_m;
    const int k_begin = split * p.k_split, k_end = min(p.K, k_begin + p.k_split);
    const bool none = EXPERTS && t.expert >= p.experts;   // pairs of no expert: zeros

    int4v acc[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
        acc[nb] = int4v{0, 0, 0, 0};

    if (!none) {
        const __amdgpu_buffer_rsrc_t w = make_rsrc(W + (int64_t)n0 * p.w_pitch,
                                                   (uint32_t)min(16 * NB, p.N - n0) * (uint32_t)p.w_pitch);
        // (experts: all of A, less than 2^31 bytes)
        const __amdgpu_buffer_rsrc_t a =
            EXPERTS ? make_rsrc(p.A, (uint32_t)p.M * (uint32_t)p.a_pitch)
                    : make_rsrc(p.A + (int64_t)t.first * p.a_pitch, (uint32_t)t.rows * (uint32_t)p.a_pitch);
        const uint32_t a_off = row < 0 ? 0x80000000u
                                       : (uint32_t)(EXPERTS ? row : i) * (uint32_t)p.a_pitch + 16u * g;
        const uint32_t w_off = (uint32_t)i * (uint32_t)p.w_pitch + 16u * g;
        struct Step {
            int4v w[NB][kChunks], a[kChunks];
        };
        const auto load = [&](int k, Step &s) {
            const uint32_t at = (uint32_t)__builtin_amdgcn_readfirstlane(k);
#pragma unroll
            for (int j = 0; j < kChunks; ++j) {
                const uint32_t gone = oob_unless(k + 64 * j + 16 * g < k_end);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                    s.w[nb][j] = __builtin_bit_cast(
                        int4v, __builtin_amdgcn_raw_buffer_load_b128(
                                   w, (w_off + (uint32_t)(16 * nb) * (uint32_t)p.w_pitch + 64u * j) | gone, at, 0));
                s.a[j] = __builtin_bit_cast(int4v, __builtin_amdgcn_raw_buffer_load_b128(a, (a_off + 64u * j) | gone, at, 0));
            }
        };
        const auto multiply = [&](const Step &s) {
#pragma unroll
            for (int j = 0; j < kChunks; ++j)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                    acc[nb] = i8_mfma(s.w[nb][j], s.a[j], acc[nb]);
        };
        constexpr int kStride = kWaves * kI8StreamK;
        const int first = k_begin + wave * kI8StreamK;
        if (first < k_end) {
            Step s[DEPTH];
#pragma unroll
            for (int d = 0; d < DEPTH; ++d)
                load(first + d * kStride, s[d]);
            for (int k = first;; k += DEPTH * kStride) {
                bool done = false;
#pragma unroll
                for (int d = 0; d < DEPTH; ++d) {
                    multiply(s[d]);
                    if (k + (d + 1) * kStride >= k_end) {
                        done = true;
                        break;
                    }
                    load(k + (d + DEPTH) * kStride, s[d]);
                }
                if (done)
                    break;
            }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
            part[wave][nb][lane] = acc[nb];
    }
    __syncthreads();

    // thread e adds up and writes columns 4 g .. + 3 of row i of block nb
    for (int e = tid; e < NB * 64; e += 64 * kWaves) {
        const int nb = e >> 6, l = e & 63;   // l & 15 == lane & 15: the row is this lane's
        const int n = n0 + 16 * nb + 4 * (l >> 4);
        if (pair < 0 || n >= p.N)
            continue;
        int4v sum = {0, 0, 0, 0};
        if (!none) {
#pragma unroll
            for (int v = 0; v < kWaves; ++v)
                sum += part[v][nb][l];
        }
        const int many = min(4, p.N - n);
        if (!EXPERTS && p.partial) {
            int *to = p.partial + ((int64_t)split * p.M + pair) * p.N + n;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r < many)
                    to[r] = sum[r];
        } else {
            const float factor = none ? 0.0f : p.alpha * p.a_scales[row];
            half_t *to = p.C + (int64_t)pair * p.N + n;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r < many)
                    to[r] = none ? (half_t)0 : i8_out(sum[r], factor, w_scales[n + r], p.relu);
        }
    }
}

} // namespace

hipError_t launch_i8_stream(const I8Args &a, int64_t grid, bool experts, hipStream_t s)
{
    if (experts)
        hipLaunchKernelGGL(i8_stream_kernel<true>, dim3((unsigned)grid), dim3(64 * kWaves), 0, s, a);
    else
        hipLaunchKernelGGL(i8_stream_kernel<false>, dim3((unsigned)grid), dim3(64 * kWaves), 0, s, a);
    return hipGetLastError();
}

// ---- the sum of a split's parts ---------------------------------------------------
// Four columns a thread where C takes 8-byte stores, else one.  Bound by memory and
// the launch: 64 x 8192 in four parts 4 us.
template <bool VEC4>
__global__ void __launch_bounds__(256) i8_reduce_kernel(I8Args p)
{
    constexpr int V = VEC4 ? 4 : 1;
    const int64_t mn = (int64_t)p.M * p.N;
    for (int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V; e < mn; e += (int64_t)gridDim.x * 256 * V) {
        const int64_t m = mn < (int64_t)1 << 31 ? (int64_t)((uint32_t)e / (uint32_t)p.N) : e / p.N, n = e - m * p.N;
        int sum[V];
#pragma unroll
        for (int r = 0; r < V; ++r)
            sum[r] = 0;
        for (int s = 0; s < p.splits; ++s) {
            const int *from = p.partial + s * mn + e;
            if constexpr (VEC4) {
                const int4v v = *reinterpret_cast<const int4v *>(from);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    sum[r] += v[r];
            } else {
                sum[0] += *from;
            }
        }
        const float factor = p.alpha * p.a_scales[m];
        half_t h[V];
#pragma unroll
        for (int r = 0; r < V; ++r)
            h[r] = i8_out(sum[r], factor, p.w_scales[n + r], p.relu);
        if constexpr (VEC4) {
            *reinterpret_cast<half4 *>(p.C + e) = half4{h[0], h[1], h[2], h[3]};
        } else {
            p.C[e] = h[0];
        }
    }
}

hipError_t launch_i8_reduce(const I8Args &a, hipStream_t s)
{
    const bool vec4 = a.vec_c >= 4;
    const int64_t items = (int64_t)a.M * a.N / (vec4 ? 4 : 1);
    const dim3 grid((unsigned)std::min<int64_t>((items + 255) / 256, 256 * 16));
    if (vec4)
        hipLaunchKernelGGL(i8_reduce_kernel<true>, grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL(i8_reduce_kernel<false>, grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

} // namespace gemm_f16_impl
