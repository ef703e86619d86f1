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
    int tiles_m, tiles_n;    // workgroups
    int splits, split_blocks;   // parts of K, k blocks of one
    float *W;                // a split's partial sums, splits x rows x N; null: unsplit
    int rows, row0;          // rows of the call, and the first of this launch
    float alpha;
    int relu;
};

struct Q4Config {
    const char *name;
    int m_blocks;            // rows of A of a workgroup, in 16s
    int n_blocks;            // rows of W of a workgroup, in 16s
    int waves;
    int stages;              // LDS stages of the tile kernel, each of 128 k; 0: the kernel for few rows
};
constexpr int kNumQ4Configs = 8;
constexpr int kQ4Expanded = 7;   // W expanded into the workspace, then the dense product
extern const Q4Config kQ4Configs[kNumQ4Configs];

// The kernel for few rows adds its waves' sums this many 16-column blocks at
// a time: 64 KiB of LDS at most.
constexpr int q4_sum_chunk(int m_blocks, int n_blocks) { return m_blocks * n_blocks <= 8 ? n_blocks : 8 / m_blocks; }
int64_t q4_lds_bytes(const Q4Config &c, int group);
// The kernel for few rows: tiles_n x tiles_m x splits workgroups.
hipError_t launch_q4(int config, int group, const Q4Args &a, hipStream_t s);
// The tile kernel: tiles_m x tiles_n x splits workgroups; A's rows 4-byte aligned.
hipError_t launch_q4_tile(int config, int group, const Q4Args &a, int64_t grid, hipStream_t s);
// A's M rows of K copied to rows of `pitch` (a multiple of 8), zeros behind them.
hipError_t launch_q4_pack(const _Float16 *A, _Float16 *to, int64_t M, int64_t K, int64_t pitch, hipStream_t s);
hipError_t launch_q4_compress(const _Float16 *W, uint32_t *codes, uint32_t *words, int64_t N, int64_t K, int group,
                              bool symmetric, hipStream_t s);
hipError_t launch_q4_expand(const uint32_t *codes, const uint32_t *words, _Float16 *W, int64_t N, int64_t K, int group,
                            hipStream_t s);

// The paged cache (include/gemm_f16_q4.h) as the kernels see it.
struct Q4Pages {
    uint32_t *k_codes, *k_words, *v_codes, *v_words;
    int64_t pages;
    int heads, page_size, head_dim, group;
    const int32_t *table;     // batch x max_pages
    int batch, max_pages;
    uint32_t page_magic;      // t / page_size = (t page_magic >> 32) >> page_shift for 0 <= t < 2^31
    int page_shift;
};

struct Q4AppendArgs {
    Q4Pages c;
    const _Float16 *K, *V, *Q;
    _Float16 *Q_out;
    int64_t k_stride, v_stride, q_stride;
    const int32_t *lengths, *starts;
    const float *cos, *sin;
    int64_t positions;
    int tokens, q_heads, rotary, interleaved;
    int vec_k, vec_v, vec_q, vec_out;   // rows are 16-byte aligned
};
hipError_t launch_q4_append(const Q4AppendArgs &a, hipStream_t s);

struct Q4ReadArgs {
    Q4Pages c;
    const int32_t *first, *starts;
    _Float16 *K, *V;
    int tokens;
};
hipError_t launch_q4_read(const Q4ReadArgs &a, hipStream_t s);

struct Q4AttentionArgs {
    Q4Pages c;
    const _Float16 *Q;
    int64_t q_stride;
    const int32_t *lengths;
    _Float16 *out;
    float *parts;             // splits > 1: batch x q_heads x splits x head_dim sums, then as many (max, sum) pairs
    float scale;
    int q_heads, ratio;       // query heads; query heads of a cache head
    int row_tiles, splits;
    int step;                 // tokens of a wave's step: 32, or 64 or 128 where up to 8 or 4 heads share the columns
};
constexpr int kQ4AttentionWaves = 4;
constexpr int kQ4AttentionTokens = 32;   // a wave's step
int64_t q4_attention_lds_bytes(int head_dim);
hipError_t launch_q4_attention(const Q4AttentionArgs &a, int64_t grid, hipStream_t s);

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

// The masks and the numbers that are OR-ed in.  v_and_or_b32 does both, but
// takes no literal and one scalar operand: the values are kept from the
// compiler's constant folding, the masks in scalar registers and the numbers
// in vector registers, or it would emit an AND and an OR with a literal each.
struct q4_bits {
    unsigned low, high, low_one, high_one;
    __device__ __forceinline__ q4_bits()
    {
        asm("s_mov_b32 %0, 0x000F000F" : "=s"(low));
        asm("s_mov_b32 %0, 0x00F000F0" : "=s"(high));
        asm("v_mov_b32 %0, 0x64006400" : "=v"(low_one));
        asm("v_mov_b32 %0, 0x54005400" : "=v"(high_one));
    }
};

// q - z of a dword's eight codes, exact, with the addends of the value pairs
// 0-1, 2-3, 4-5 and 6-7: nine instructions.
__device__ __forceinline__ q4_half8 q4_codes(unsigned w, const q4_bits &m, unsigned z0, unsigned z1, unsigned z2, unsigned z3)
{
    const q4_half2 p0 = q4_pair((w & m.low) | m.low_one, z0);
    const q4_half2 p1 = q4_pair((w & m.high) | m.high_one, z1);
    w >>= 8;
    const q4_half2 p2 = q4_pair((w & m.low) | m.low_one, z2);
    const q4_half2 p3 = q4_pair((w & m.high) | m.high_one, z3);
    return q4_half8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}
__device__ __forceinline__ q4_half8 q4_codes(unsigned w, const q4_bits &m, const q4_zero &z)
{
    return q4_codes(w, m, z.a, z.b, z.a, z.b);
}

// 64 + q of a dword's eight codes: seven instructions, for products whose sum
// of the other operand is known and takes the 64 off again.
__device__ __forceinline__ q4_half8 q4_codes_64(unsigned w, const q4_bits &m)
{
    const q4_half2 p0 = __builtin_bit_cast(q4_half2, (w << 4 & m.high) | m.high_one);
    const q4_half2 p1 = __builtin_bit_cast(q4_half2, (w & m.high) | m.high_one);
    const q4_half2 p2 = __builtin_bit_cast(q4_half2, (w >> 4 & m.high) | m.high_one);
    const q4_half2 p3 = __builtin_bit_cast(q4_half2, (w >> 8 & m.high) | m.high_one);
    return q4_half8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

__device__ __forceinline__ float q4_scale(unsigned word)
{
    return (float)__builtin_bit_cast(q4_half2, word)[0];
}

// x / s, correctly rounded, for an s of at most 11 bits whose reciprocal is r
// to within an ulp or two: the remainder of x r is exact, and with it the
// quotient is known to 2^-44 of itself, while a quotient of 24 bits by 11 is at
// least 2^-36 of itself away from every number half way between two floats
// (never on one: that number times s would need 25 bits).  Not for infinite
// x; where the remainder underflows the quotient is nothing next to 1/2.
__device__ __forceinline__ float q4_divide(float x, float s, float r)
{
    const float q = x * r;
    return __builtin_fmaf(__builtin_fmaf(-s, q, x), r, q);
}

// Scale word and codes of a group, from its extreme values.  NaN has been
// replaced by 0 before.
struct q4_rounder {
    static constexpr float kLarge = 3e38f;                // for infinite values
    static constexpr float kInteger = 12582912.0f;        // 1.5 2^23: its neighbours are 1 apart
    float s, z, r;
    __device__ __forceinline__ q4_rounder(float lo, float hi, bool symmetric)
    {
        lo = __builtin_fminf(lo, 0.0f);
        hi = __builtin_fmaxf(hi, 0.0f);
        // infinity becomes NaN here, which the minimum takes for 65504
        const float wide = symmetric ? q4_divide(__builtin_fmaxf(hi, -lo), 7.0f, 1.0f / 7.0f)
                                     : q4_divide(hi - lo, 15.0f, 1.0f / 15.0f);
        s = (float)(_Float16)__builtin_fminf(__builtin_fabsf(wide), 65504.0f);   // |.|: never -0
        r = s > 0.0f ? __builtin_amdgcn_rcpf(s) : 0.0f;
        z = symmetric ? 8.0f
                      : __builtin_amdgcn_fmed3f(__builtin_rintf(q4_divide(__builtin_fminf(-lo, kLarge), s, r)), 0.0f, 15.0f);
    }
    __device__ __forceinline__ unsigned word() const
    {
        const _Float16 h = (_Float16)s;
        return (unsigned)__builtin_bit_cast(unsigned short, h) | (unsigned)z << 16;
    }

    // Codes come as the bits of kInteger + n, with n = code - z: the sum rounds
    // to an integer as rint does (halves to even).
    __device__ __forceinline__ unsigned clamped(float t) const
    {
        return __builtin_bit_cast(unsigned, __builtin_amdgcn_fmed3f(t, kInteger - z, kInteger + 15.0f - z));
    }
    // of any x
    __device__ __forceinline__ unsigned code(float x) const
    {
        return clamped(q4_divide(__builtin_amdgcn_fmed3f(x, -kLarge, kLarge), s, r) + kInteger);
    }
    // Of a binary16 x, without the remainder: for x and s of 11 bits the
    // quotient either is a multiple of 1/2 or at least 2^-13 from one (where it
    // matters, between codes), and x r is within 2^-17 of it, so rounding x r to
    // a multiple of 2^-14 (adding 768) puts it on the multiple or leaves it on
    // its side.  Taking the 768 off is exact and part of the second sum.
    __device__ __forceinline__ unsigned code16(float x) const
    {
        return clamped(__builtin_fmaf(x, r, 768.0f) + (kInteger - 768.0f));
    }
    // The dword of eight codes: their bits summed at the codes' places, in which
    // nothing carries once the constant part is taken off.
    __device__ __forceinline__ unsigned join(const unsigned (&bits)[8]) const
    {
        unsigned dw = ((unsigned)z - 0x4B400000u) * 0x11111111u;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            dw += bits[i] << (4 * (i / 2 + 4 * (i & 1)));
        return dw;
    }
};

// Smallest lo and largest hi of neighbouring lanes, 2, 4, 8 or 16 of a row.
template <int LANES>
__device__ __forceinline__ void q4_row_extremes(float &lo, float &hi)
{
    const auto with = [&](float l, float h) {
        lo = __builtin_fminf(lo, l);
        hi = __builtin_fmaxf(hi, h);
    };
#define GEMM_F16_Q4_DPP(x, ctrl) \
    __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), ctrl, 0xF, 0xF, true))
    with(GEMM_F16_Q4_DPP(lo, 0xB1), GEMM_F16_Q4_DPP(hi, 0xB1));             // the lane next to it
    if constexpr (LANES > 2)
        with(GEMM_F16_Q4_DPP(lo, 0x4E), GEMM_F16_Q4_DPP(hi, 0x4E));         // the other pair of four
    if constexpr (LANES > 4)
        with(GEMM_F16_Q4_DPP(lo, 0x141), GEMM_F16_Q4_DPP(hi, 0x141));       // eight mirrored: the other four
    if constexpr (LANES > 8)
        with(GEMM_F16_Q4_DPP(lo, 0x140), GEMM_F16_Q4_DPP(hi, 0x140));       // sixteen mirrored: the other eight
#undef GEMM_F16_Q4_DPP
}

// ... of the four lanes 16 and 32 apart.  The swaps exchange rows of 16 or
// halves of 32 lanes between two registers; of two copies of x they leave
// each pair's values side by side.
__device__ __forceinline__ void q4_column_extremes(float &lo, float &hi)
{
    const auto pair16 = [](float x, auto pick) {
        const unsigned v = __builtin_bit_cast(unsigned, x);
        const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return pick(__builtin_bit_cast(float, (unsigned)a[0]), __builtin_bit_cast(float, (unsigned)a[1]));
    };
    const auto pair32 = [](float x, auto pick) {
        const unsigned v = __builtin_bit_cast(unsigned, x);
        const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return pick(__builtin_bit_cast(float, (unsigned)a[0]), __builtin_bit_cast(float, (unsigned)a[1]));
    };
    const auto least = [](float a, float b) { return __builtin_fminf(a, b); };
    const auto most = [](float a, float b) { return __builtin_fmaxf(a, b); };
    lo = pair32(pair16(lo, least), least);
    hi = pair32(pair16(hi, most), most);
}

// LDS written by a wave is read by the same wave: its LDS accesses complete in
// order, the compiler must only keep them so.
__device__ __forceinline__ void q4_wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Position of value i of eight in a dword, in bits.
__device__ __forceinline__ constexpr int q4_shift(int i) { return 4 * (i / 2 + 4 * (i & 1)); }

// ---- the paged cache ---------------------------------------------------------------
// Index in the page table of position t, 0 <= t < 2^31.
__device__ __forceinline__ int q4_page_of(const Q4Pages &c, int t)
{
    return (int)(__umulhi((uint32_t)t, c.page_magic) >> c.page_shift);
}

// Page of the granule of 8 tokens that holds position pos of sequence b, or -1
// where the table or the pool has none.
__device__ __forceinline__ int q4_page(const Q4Pages &c, int b, int64_t pos)
{
    if (pos < 0 || pos >= (int64_t)c.max_pages * c.page_size)
        return -1;
    const int id = c.table[(int64_t)b * c.max_pages + q4_page_of(c, (int)pos)];
    return id >= 0 && id < c.pages ? id : -1;
}

// Work of an append or a read: a granule is 8 positions, a multiple of 8 on,
// that one wave handles for one head (a dword of v_codes holds the 8 tokens
// of one d, so nobody else may write it).  n rows of a sequence touch at most
// n / 8 + 2 granules, so units starts[b] / 8 + 2 b up to the next sequence's
// are enough for sequence b; the rest of them is empty.
struct q4_granule {
    int b, row, slot, count;   // sequence, first row, its slot in the granule, rows
    int64_t pos;               // position of slot 0
};

__device__ __forceinline__ q4_granule q4_find(int64_t unit, const int32_t *starts, const int32_t *first, int tokens,
                                              int batch)
{
    q4_granule r = {0, 0, 0, 0, 0};
    int lo = 0, row0, rows;
    int64_t local;
    if (!starts) {             // one row for each sequence
        lo = row0 = (int)unit;
        rows = 1;
        local = 0;
    } else {
        // the last sequence whose units begin at or before this one: 64 at a time
        const int lane = threadIdx.x & 63;
        for (int n = batch; n > 1;) {
            const int step = (n + 63) / 64;
            const bool before = lane * step < n && starts[lo + lane * step] / 8 + 2 * (int64_t)(lo + lane * step) <= unit;
            const int k = __popcll(__ballot(before)) - 1;
            if (k < 0)
                return r;
            n = min(step, n - k * step);
            lo += k * step;
        }
        row0 = min(max(starts[lo], 0), tokens);
        rows = min(max(starts[lo + 1], row0), tokens) - row0;
        local = unit - (starts[lo] / 8 + 2 * (int64_t)lo);
        if (local < 0)
            return r;
    }
    const int64_t p0 = first ? first[lo] : 0, granule = (p0 >= 0 ? p0 / 8 : -((7 - p0) / 8)) + local;
    const int64_t begin = p0 > granule * 8 ? p0 : granule * 8, end = p0 + rows < granule * 8 + 8 ? p0 + rows : granule * 8 + 8;
    r.b = lo;
    r.pos = granule * 8;
    r.row = (int)(row0 + (begin - p0));
    r.slot = (int)(begin - granule * 8);
    r.count = begin < end ? (int)(end - begin) : 0;
    return r;
}

// Place of the dword of d = 8 c .. 8 c + 7 in a token's row of k_codes.
template <int D>
__device__ __forceinline__ int q4_key_dword(int c)
{
    constexpr int B = D < 128 ? D : 128;
    const int in = c % (B / 8);
    return c / (B / 8) * (B / 8) + in % 4 * (B / 32) + in / 4;
}

#endif // __HIPCC__

} // namespace gemm_f16_impl

#endif
