// gemm_f16_q4_format.h -- the 4-bit operand format on the device (the format
// itself is described in include/gemm_f16_q4.h) and the launchers of its
// kernels.  Not part of the public ABI.
#ifndef GEMM_F16_Q4_FORMAT_H
#define GEMM_F16_Q4_FORMAT_H

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gemm_f16_impl {

// ---- launchers -----------------------------------------------------------------
struct Q4Args {
    const _Float16 *A;       // M x K
    const uint32_t *codes;   // [NB][KB][64 lanes][4]
    const uint32_t *words;   // [NB][KB][16][128 / group]
    _Float16 *C;             // M x N
    int M, N, K;
    int n_blocks, k_blocks;  // tiles of 16 rows of W, of 128 k
    int chunk;               // k staged in LDS at a time, a multiple of 128 waves
    int vec_a;               // A's rows are 16-byte aligned
    float alpha;
    int relu;
};

struct Q4Config {
    const char *name;
    int m_blocks;            // rows of A of a workgroup, in 16s
    int n_blocks;            // rows of W of a workgroup, in 16s
    int waves;               // they share the workgroup's k blocks in turn
};
constexpr int kNumQ4Configs = 3;
extern const Q4Config kQ4Configs[kNumQ4Configs];

int64_t q4_lds_bytes(const Q4Config &c, int64_t M, int chunk);
int q4_chunk(const Q4Config &c, int64_t M, int64_t K);
hipError_t launch_q4(int config, int group, const Q4Args &a, int64_t grid_n, int64_t grid_m, hipStream_t s);
hipError_t launch_q4_compress(const _Float16 *W, uint32_t *codes, uint32_t *words, int64_t N, int64_t K, int group,
                              bool symmetric, bool vec, hipStream_t s);
hipError_t launch_q4_expand(const uint32_t *codes, const uint32_t *words, _Float16 *W, int64_t N, int64_t K, int group,
                            bool vec, hipStream_t s);

#ifdef __HIPCC__

typedef _Float16 q4_half2 __attribute__((ext_vector_type(2)));
typedef _Float16 q4_half8 __attribute__((ext_vector_type(8)));
typedef unsigned q4_uint4 __attribute__((ext_vector_type(4)));
typedef float q4_float4 __attribute__((ext_vector_type(4)));

// A binary16 with 10 mantissa bits read as an integer: 0x6400 | q is 1024 + q,
// and 0x5400 | q << 4 is 64 + q, both exact, so that a masked nibble becomes
// a number with one OR.  Adding -(1024 + z) or -(64 + z), exact too, leaves
// q - z.  q4_zero holds those two addends, each twice.
struct q4_zero {
    unsigned a, b;
    __device__ __forceinline__ explicit q4_zero(unsigned word)
    {
        const unsigned zz = (word >> 16) * 0x10001u;
        a = zz | 0xE400E400u;
        b = zz << 4 | 0xD400D400u;
    }
    __device__ __forceinline__ q4_zero(unsigned z0, unsigned z1)   // zero points of the two halves
    {
        const unsigned zz = z0 | z1 << 16;
        a = zz | 0xE400E400u;
        b = zz << 4 | 0xD400D400u;
    }
};

__device__ __forceinline__ q4_half2 q4_pair(unsigned bits, unsigned zero)
{
    return __builtin_bit_cast(q4_half2, bits) + __builtin_bit_cast(q4_half2, zero);
}

// q - z of a dword's eight codes, exact: nine instructions.
__device__ __forceinline__ q4_half8 q4_codes(unsigned w, const q4_zero &z)
{
    const q4_half2 p0 = q4_pair((w & 0x000F000Fu) | 0x64006400u, z.a);
    const q4_half2 p1 = q4_pair((w & 0x00F000F0u) | 0x54005400u, z.b);
    w >>= 8;
    const q4_half2 p2 = q4_pair((w & 0x000F000Fu) | 0x64006400u, z.a);
    const q4_half2 p3 = q4_pair((w & 0x00F000F0u) | 0x54005400u, z.b);
    return q4_half8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

__device__ __forceinline__ float q4_scale(unsigned word)
{
    return (float)__builtin_bit_cast(q4_half2, word)[0];
}

// Scale word and codes of a group, from its extreme values; no contraction
// to fused multiply-adds, so that the results are those of the formulas.
struct q4_rounder {
    float s, z;
    __device__ __forceinline__ q4_rounder(float lo, float hi, bool symmetric)
    {
        lo = __builtin_fminf(lo, 0.0f);
        hi = __builtin_fmaxf(hi, 0.0f);
        const float wide = symmetric ? __builtin_fmaxf(hi, -lo) / 7.0f : (hi - lo) / 15.0f;
        s = (float)(_Float16)__builtin_fminf(__builtin_fabsf(wide), 65504.0f);   // |.|: never -0
        z = symmetric ? 8.0f : s > 0.0f ? __builtin_fminf(__builtin_fmaxf(__builtin_rintf(-lo / s), 0.0f), 15.0f) : 0.0f;
    }
    __device__ __forceinline__ unsigned word() const
    {
        const _Float16 h = (_Float16)s;
        return (unsigned)__builtin_bit_cast(unsigned short, h) | (unsigned)z << 16;
    }
    __device__ __forceinline__ unsigned code(float x) const
    {
        const float t = s > 0.0f ? __builtin_rintf(x / s) : 0.0f;
        return (unsigned)__builtin_fminf(__builtin_fmaxf(t + z, 0.0f), 15.0f);
    }
};

// Position of value i of eight in a dword, in bits.
__device__ __forceinline__ constexpr int q4_shift(int i) { return 4 * (i / 2 + 4 * (i & 1)); }

#endif // __HIPCC__

} // namespace gemm_f16_impl

#endif
