// gemm_f16_i8_rows.hip -- rows of binary16 to 8-bit codes and back, and the
// weighted sum of the experts' results: kernels that read and write each
// element once and are bound by memory.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gemm_f16_i8_internal.h"

namespace gemm_f16_impl {

namespace {

typedef _Float16 half_t;
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef half8 half8_any __attribute__((aligned(2)));   // 16-byte accesses at any element's address
typedef int int4v __attribute__((ext_vector_type(4)));
typedef float float4v __attribute__((ext_vector_type(4)));

// Sixteen elements of a row from column c on, zeros past K.
__device__ __forceinline__ void load16(const half_t *row, int64_t K, int64_t c, half_t (&x)[16])
{
    if (c + 16 <= K) {
        const half8 lo = *reinterpret_cast<const half8_any *>(row + c), hi = *reinterpret_cast<const half8_any *>(row + c + 8);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = lo[i];
            x[8 + i] = hi[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            x[i] = c + i < K ? row[c + i] : (half_t)0;
    }
}

// NaN as 0, infinities as 65504
__device__ __forceinline__ float finite(half_t x)
{
    const float f = (float)x;
    return f != f ? 0.0f : __builtin_fminf(__builtin_fmaxf(f, -65504.0f), 65504.0f);
}

// rint(127 x / m) for binary16 |x| <= m.  t = 127 x is exact in fp32 (18 bits).
// y is the quotient but for 2^-22 of itself; r = t - y m is exact (at most 2^-22
// of t, on a grid of 2^-33 of it), so y + r / m is the quotient but for 2^-46 of
// itself, rounded once to fp32: exactly the half where the quotient is one.  Any
// other quotient near a half h in 2^(6 - e) .. 2^(7 - e) differs from it by at least
// 2^-(11 + e) (an integer over m's 11 bits, shifted by as much as x is smaller),
// while half a step of fp32 there is 2^-(18 + e).
__device__ __forceinline__ int code_of(float x, float m, float inverse)
{
    const float t = 127.0f * x;
    float y = t * inverse;
    y = __builtin_fmaf(__builtin_fmaf(-y, m, t), inverse, y);
    return (int)__builtin_rintf(y);
}

// THREADS threads take a row, 16 elements each at a time; up to HELD of those stay
// in registers between the search for the largest magnitude and the rounding,
// longer rows are read again.  Bound by memory where rows are many (8192 x 8192 37 us
// from memory, 5.4 TB/s; 32 where X is still in a cache), else by the latency of load,
// search and store (13 x 4100 4.1 us).
constexpr int block_of(int threads) { return threads > 256 ? threads : 256; }
template <int THREADS, int HELD>
__global__ void __launch_bounds__(block_of(THREADS)) i8_compress_kernel(const half_t *__restrict__ X, int64_t stride, int8_t *__restrict__ codes,
                                                          int64_t pitch, float *__restrict__ scales, int64_t rows, int64_t K)
{
    constexpr int ROWS = block_of(THREADS) / THREADS, WAVES = block_of(THREADS) / 64;
    __shared__ float most_of[WAVES];
    const int t = threadIdx.x % THREADS;
    const int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / THREADS;
    if (THREADS <= 64 && r >= rows)
        return;
    const half_t *row = X + r * stride;
    half_t x[HELD][16];
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        const int64_t c = 16 * (int64_t)(t + i * THREADS);
        if (c < K) {
            load16(row, K, c, x[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                x[i][j] = (half_t)0;
        }
    }
#pragma unroll
    for (int i = 0; i < HELD; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j)
            m = __builtin_fmaxf(m, __builtin_fabsf(finite(x[i][j])));
    for (int64_t c = 16 * (int64_t)(t + HELD * THREADS); c < K; c += 16 * THREADS) {
        half_t y[16];
        load16(row, K, c, y);
#pragma unroll
        for (int j = 0; j < 16; ++j)
            m = __builtin_fmaxf(m, __builtin_fabsf(finite(y[j])));
    }
#pragma unroll
    for (int d = 1; d < (THREADS < 64 ? THREADS : 64); d *= 2)
        m = __builtin_fmaxf(m, __shfl_xor(m, d));
    if constexpr (THREADS > 64) {
        if (threadIdx.x % 64 == 0)
            most_of[threadIdx.x / 64] = m;
        __syncthreads();
        m = most_of[0];
#pragma unroll
        for (int w = 1; w < WAVES; ++w)
            m = __builtin_fmaxf(m, most_of[w]);
    }
    const float inverse = m > 0.0f ? 1.0f / m : 0.0f;
    if (t == 0)
        scales[r] = m / 127.0f;
    const auto put = [&](int64_t c, const half_t (&y)[16]) {
        int4v v;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            int packed = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                packed |= (code_of(finite(y[4 * w + b]), m, inverse) & 255) << (8 * b);
            v[w] = packed;
        }
        *reinterpret_cast<int4v *>(codes + r * pitch + c) = v;
    };
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        const int64_t c = 16 * (int64_t)(t + i * THREADS);
        if (c < pitch)
            put(c, x[i]);
    }
    for (int64_t c = 16 * (int64_t)(t + HELD * THREADS); c < pitch; c += 16 * THREADS) {
        half_t y[16];
        load16(row, K, c, y);
        put(c, y);
    }
}

// i / n for 0 <= i < items, n >= 1: in 32 bits where those do, a 64-bit division takes longer than the rest of a small kernel.
__device__ __forceinline__ int64_t quotient(int64_t i, int64_t n, int64_t items)
{
    return items < (int64_t)1 << 31 ? (int64_t)((uint32_t)i / (uint32_t)n) : i / n;
}

// Sixteen codes of a row a thread.  Bound by memory: 8192 x 8192 39 us, 5.2 TB/s; 30 where the codes were just written.
__global__ void __launch_bounds__(256) i8_expand_kernel(const int8_t *__restrict__ codes, int64_t pitch,
                                                        const float *__restrict__ scales, half_t *__restrict__ X, int64_t items,
                                                        int64_t K, int64_t per_row)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < items; i += (int64_t)gridDim.x * 256) {
        const int64_t r = quotient(i, per_row, items), c = (i - r * per_row) * 16;
        const int4v v = *reinterpret_cast<const int4v *>(codes + r * pitch + c);
        const float s = scales[r];
        half_t x[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            x[j] = (half_t)(s * (float)((int)((unsigned)v[j / 4] << (24 - 8 * (j % 4))) >> 24));
        half_t *to = X + r * K + c;
        if (c + 16 <= K) {
            *reinterpret_cast<half8_any *>(to) = half8{x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]};
            *reinterpret_cast<half8_any *>(to + 8) = half8{x[8], x[9], x[10], x[11], x[12], x[13], x[14], x[15]};
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (c + j < K)
                    to[j] = x[j];
        }
    }
}

// V columns of a token's sum a thread, in fp32 and in the order of the slots,
// the results of eight slots in flight (1 token of 8 x 2048: 4.8 us one after the other, 3.4).
template <int V>
__global__ void __launch_bounds__(256) expert_sum_kernel(const half_t *__restrict__ Y, const float *__restrict__ weights,
                                                         half_t *__restrict__ out, int64_t items, int top_k, int64_t N,
                                                         int64_t per_row)
{
    typedef _Float16 vec __attribute__((ext_vector_type(V)));
    typedef vec vec_any __attribute__((aligned(2)));
    constexpr int AHEAD = 8;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < items; i += (int64_t)gridDim.x * 256) {
        const int64_t t = quotient(i, per_row, items), c = (i - t * per_row) * V;
        const half_t *from = Y + t * top_k * N + c;
        const float *w = weights + t * top_k;
        const int n = (int)(N - c < V ? N - c : V);
        float sum[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
            sum[e] = 0.0f;
        if (n == V) {
            for (int j0 = 0; j0 < top_k; j0 += AHEAD) {
                vec y[AHEAD];
                float wj[AHEAD];
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    const int at = min(j0 + j, top_k - 1);   // (again the last one: not added)
                    y[j] = *reinterpret_cast<const vec_any *>(from + (int64_t)at * N);
                    wj[j] = w[at];
                }
#pragma unroll
                for (int j = 0; j < AHEAD; ++j)
                    if (j0 + j < top_k) {
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            sum[e] = __builtin_fmaf(wj[j], (float)y[j][e], sum[e]);
                    }
            }
        } else {
            for (int j = 0; j < top_k; ++j)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (e < n)
                        sum[e] = __builtin_fmaf(w[j], (float)from[(int64_t)j * N + e], sum[e]);
        }
        half_t *to = out + t * N + c;
        if (n == V) {
            vec h;
#pragma unroll
            for (int e = 0; e < V; ++e)
                h[e] = (half_t)sum[e];
            *reinterpret_cast<vec_any *>(to) = h;
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (e < n)
                    to[e] = (half_t)sum[e];
        }
    }
}

unsigned blocks_for(int64_t items) { return (unsigned)std::min<int64_t>((items + 255) / 256, 256 * 32); }

} // namespace

hipError_t launch_i8_compress(const _Float16 *X, int64_t stride, int8_t *codes, int64_t pitch, float *scales, int64_t rows,
                              int64_t K, hipStream_t s)
{
    constexpr int64_t most = 1 << 21;   // rows of a launch: its work items are counted in 32 bits
    for (; rows > most; rows -= most) {
        const hipError_t e = launch_i8_compress(X, stride, codes, pitch, scales, most, K, s);
        if (e != hipSuccess)
            return e;
        X += most * stride;
        codes += most * pitch;
        scales += most;
    }
    if (K <= 256)
        hipLaunchKernelGGL((i8_compress_kernel<16, 1>), dim3((unsigned)((rows + 15) / 16)), dim3(256), 0, s, X, stride, codes,
                           pitch, scales, rows, K);
    else if (K <= 2048)
        hipLaunchKernelGGL((i8_compress_kernel<64, 2>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, s, X, stride, codes,
                           pitch, scales, rows, K);
    else if (K <= 8192)
        hipLaunchKernelGGL((i8_compress_kernel<256, 2>), dim3((unsigned)rows), dim3(256), 0, s, X, stride, codes, pitch, scales,
                           rows, K);
    else if (K <= 16384 && rows >= 256)   // (8192 x 14336: 73 us, 1024 threads 110)
        hipLaunchKernelGGL((i8_compress_kernel<256, 4>), dim3((unsigned)rows), dim3(256), 0, s, X, stride, codes, pitch, scales,
                           rows, K);
    else   // (1 x 28672: 256 threads, which hold 8192 elements, 7.8 us; 5.6 so)
        hipLaunchKernelGGL((i8_compress_kernel<1024, 2>), dim3((unsigned)rows), dim3(1024), 0, s, X, stride, codes, pitch, scales,
                           rows, K);
    return hipGetLastError();
}

hipError_t launch_i8_expand(const int8_t *codes, int64_t pitch, const float *scales, _Float16 *X, int64_t rows, int64_t K,
                            hipStream_t s)
{
    const int64_t per_row = (K + 15) / 16, items = rows * per_row;
    hipLaunchKernelGGL(i8_expand_kernel, dim3(blocks_for(items)), dim3(256), 0, s, codes, pitch, scales, X, items, K, per_row);
    return hipGetLastError();
}

hipError_t launch_expert_sum(const _Float16 *Y, const float *weights, _Float16 *out, int64_t tokens, int top_k, int64_t N,
                             hipStream_t s)
{
    // two columns a thread where eight would leave CUs without work
    const int v = tokens * N < 256 * 256 * 8 ? 2 : 8;
    const int64_t per_row = (N + v - 1) / v, items = tokens * per_row;
    if (v == 2)
        hipLaunchKernelGGL(expert_sum_kernel<2>, dim3(blocks_for(items)), dim3(256), 0, s, Y, weights, out, items, top_k, N, per_row);
    else
        hipLaunchKernelGGL(expert_sum_kernel<8>, dim3(blocks_for(items)), dim3(256), 0, s, Y, weights, out, items, top_k, N, per_row);
    return hipGetLastError();
}

} // namespace gemm_f16_impl
