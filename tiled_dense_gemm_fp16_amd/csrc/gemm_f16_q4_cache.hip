// gemm_f16_q4_cache.hip -- the 4-bit paged key/value cache: appending new
// tokens (rotating keys and queries on the way) and reading tokens back.
#include <algorithm>

#include "gemm_f16_q4_format.h"
#include "gemm_f16_tile.h"

namespace gemm_f16_impl {

// A wave handles one granule of up to 8 tokens of some heads.  D / 8 lanes hold
// a token's 8-element chunks, so a pass covers 64 / (D / 8) tokens.  Groups
// reduce over group / 8 neighbouring lanes.  Keys store one dword a lane;
// values exchange codes through LDS (bytes, [token][d]) so that each lane then
// stores dwords of 8 tokens of one d.
//
// A granule's sequence, position and page take three reads one after the
// other, each as long as the reads of its tokens: with few granules every head
// has a wave of its own, and with many a wave takes several heads of one
// granule (about 4096 waves; prompts of up to 1021 tokens of 5 sequences, 48 heads of 128,
// appended and read back: 30.1 us, 31.0 with 8192 waves, 34.6 with a wave for
// every head, 37.9 with 2048; 256 sequences of one token, 80 heads: 32.4, 30.5, 44.1, 40.3).  That
// is 75 % of the rate of a copy for the prompts; 64 single tokens (5.7 us to append,
// 4.2 without starts, 6.1 to read) wait for a chain of reads: the length, the page,
// the row (which needs neither without starts) and a value's old codes (which need
// the page only).
constexpr int kCacheWaves = 4;

__device__ __forceinline__ half8 load8(const half_t *p, bool vec)
{
    if (vec)
        return *reinterpret_cast<const half8 *>(p);
    half8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = p[i];
    return v;
}

// Elements 8 c .. 8 c + 7 of a head's row, rotated; each product and sum is
// rounded by itself (no fused multiply-adds), as the formula is written.
__device__ __forceinline__ void load_rotated(const half_t *row, int c, bool vec, const Q4AppendArgs &a, int64_t pos,
                                             float x[8])
{
#pragma clang fp contract(off)
    const half8 v = load8(row + 8 * c, vec);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = (float)v[i];
    if (8 * c >= a.rotary)
        return;
    const int half = a.rotary / 2;
    const float *cs = a.cos + pos * half, *sn = a.sin + pos * half;
    if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float co = cs[4 * c + i / 2], si = sn[4 * c + i / 2], p = x[i], q = x[i + 1];
            const float pc = p * co, qs = q * si, qc = q * co, ps = p * si;
            x[i] = pc - qs;
            x[i + 1] = qc + ps;
        }
    } else {
        const bool lower = 8 * c < half;
        const half8 w = load8(row + 8 * c + (lower ? half : -half), vec);
        const int at = 8 * c - (lower ? 0 : half);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float co = cs[at + i], si = sn[at + i], own = x[i] * co, other = (float)w[i] * si;
            x[i] = lower ? own - other : own + other;
        }
    }
}

// x's codes as a dword and the group's word (the same in all its lanes);
// half: x holds binary16 values.
template <int GROUP>
__device__ __forceinline__ unsigned round_chunk(float x[8], unsigned &word, bool half)
{
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = x[i] == x[i] ? x[i] : 0.0f;
        lo = __builtin_fminf(lo, x[i]);
        hi = __builtin_fmaxf(hi, x[i]);
    }
    q4_row_extremes<GROUP / 8>(lo, hi);
    const q4_rounder r(lo, hi, false);
    word = r.word();
    unsigned bits[8];
    if (half) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            bits[i] = r.code16(x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            bits[i] = r.code(x[i]);
    }
    return r.join(bits);
}

template <int D, int GROUP>
__global__ void __launch_bounds__(64 * kCacheWaves) q4_append_kernel(Q4AppendArgs a)
{
    constexpr int LANES = D / 8, TOKENS = 64 / LANES;   // lanes of a token, tokens of a pass
    __shared__ unsigned codes[kCacheWaves][8][LANES];   // [slot][chunk]: a dword of 8 codes of the chunk
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, chunk = lane % LANES;
    const int H = a.c.heads, jobs = 2 * H + (a.Q ? a.q_heads : 0);
    const q4_granule gr = q4_find(blockIdx.x, a.starts, a.lengths, a.tokens, a.c.batch);
    if (gr.count == 0)
        return;
    const int page = q4_page(a.c, gr.b, gr.pos);
    const int in_page = page >= 0 ? (int)gr.pos - q4_page_of(a.c, (int)gr.pos) * a.c.page_size : 0;
    // positions a rotation table covers (all without one); a negative
    // position has no page
    const int64_t covered = a.cos ? a.positions : INT64_MAX;

    for (int job = blockIdx.y * kCacheWaves + wave; job < jobs; job += gridDim.y * kCacheWaves) {
        if (job >= 2 * H) {   // queries
            const int h = job - 2 * H;
#pragma unroll
            for (int pass = 0; pass < 8 / TOKENS; ++pass) {
                const int slot = pass * TOKENS + lane / LANES, row = gr.row + slot - gr.slot;
                if (slot < gr.slot || slot >= gr.slot + gr.count)
                    continue;
                float x[8] = {};
                if (page >= 0 && gr.pos + slot < covered)
                    load_rotated(a.Q + row * a.q_stride + h * D, chunk, a.vec_q, a, gr.pos + slot, x);
                half8 v;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = (half_t)x[i];
                half_t *to = a.Q_out + ((int64_t)row * a.q_heads + h) * D + 8 * chunk;
                if (a.vec_out) {
                    *reinterpret_cast<half8 *>(to) = v;
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        to[i] = v[i];
                }
            }
            continue;
        }
        if (page < 0)
            continue;
        const bool value = job >= H;
        const int h = value ? job - H : job;
        const int64_t head = (int64_t)page * H + h;
        unsigned keep = 0;   // slots of the granule that are written
#pragma unroll
        for (int pass = 0; pass < 8 / TOKENS; ++pass) {
            const int slot = pass * TOKENS + lane / LANES, row = gr.row + slot - gr.slot;
            const bool mine = slot >= gr.slot && slot < gr.slot + gr.count && gr.pos + slot < covered;
            float x[8] = {};
            if (mine) {
                if (value) {
                    const half8 v = load8(a.V + row * a.v_stride + h * D + 8 * chunk, a.vec_v);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        x[i] = (float)v[i];
                } else {
                    load_rotated(a.K + row * a.k_stride + h * D, chunk, a.vec_k, a, gr.pos + slot, x);
                }
            }
            unsigned word;
            const unsigned dw = round_chunk<GROUP>(x, word, value);
            if (mine) {
                uint32_t *words = value ? a.c.v_words : a.c.k_words;
                if (chunk % (GROUP / 8) == 0)
                    words[(head * (D / GROUP) + chunk / (GROUP / 8)) * a.c.page_size + in_page + slot] = word;
                if (!value)
                    a.c.k_codes[(head * a.c.page_size + in_page + slot) * (D / 8) + q4_key_dword<D>(chunk)] = dw;
            }
            if (value)
                codes[wave][slot][chunk] = dw;
        }
        if (!value)
            continue;
        q4_wave_fence();
#pragma unroll
        for (int s = 0; s < 8; ++s)
            if (s >= gr.slot && s < gr.slot + gr.count && gr.pos + s < covered)
                keep |= 15u << q4_shift(s);
        uint32_t *to = a.c.v_codes + (head * (a.c.page_size / 8) + in_page / 8) * D;
#pragma unroll
        for (int e = lane; e < D; e += 64) {   // in the order of the stored dwords: [d % 16][d / 16]
            const int d = e % (D / 16) * 16 + e / (D / 16);
            unsigned dw = 0;
#pragma unroll
            for (int s = 0; s < 8; ++s)
                dw |= (codes[wave][s][d / 8] >> (4 * (d % 8 / 2 + 4 * (d & 1))) & 15u) << q4_shift(s);
            to[e] = keep == 0xFFFFFFFFu ? dw : (to[e] & ~keep) | (dw & keep);   // other tokens' codes stay
        }
        q4_wave_fence();   // the next job's codes come after this one's reads
    }
}

template <int D, int GROUP>
__global__ void __launch_bounds__(64 * kCacheWaves) q4_read_kernel(Q4ReadArgs a)
{
    constexpr int LANES = D / 8, TOKENS = 64 / LANES;
    __shared__ unsigned codes[kCacheWaves][D];   // a granule's values: dword of d
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, chunk = lane % LANES;
    const int H = a.c.heads;
    const q4_granule gr = q4_find(blockIdx.x, a.starts, a.first, a.tokens, a.c.batch);
    if (gr.count == 0)
        return;
    const int page = q4_page(a.c, gr.b, gr.pos);
    const int in_page = page >= 0 ? (int)gr.pos - q4_page_of(a.c, (int)gr.pos) * a.c.page_size : 0;
    for (int job = blockIdx.y * kCacheWaves + wave; job < 2 * H; job += gridDim.y * kCacheWaves) {
        const bool value = job >= H;
        const int h = value ? job - H : job;
        const int64_t head = (int64_t)page * H + h;
        if (value && page >= 0) {
            const uint32_t *from = a.c.v_codes + (head * (a.c.page_size / 8) + in_page / 8) * D;
#pragma unroll
            for (int e = lane; e < D; e += 64)
                codes[wave][e % (D / 16) * 16 + e / (D / 16)] = from[e];
            q4_wave_fence();
        }
#pragma unroll
        for (int pass = 0; pass < 8 / TOKENS; ++pass) {
            const int slot = pass * TOKENS + lane / LANES, row = gr.row + slot - gr.slot;
            if (slot < gr.slot || slot >= gr.slot + gr.count)
                continue;
            half8 v = {};
            if (page >= 0) {
                const uint32_t *words = value ? a.c.v_words : a.c.k_words;
                const unsigned word = words[(head * (D / GROUP) + chunk / (GROUP / 8)) * a.c.page_size + in_page + slot];
                const float s = q4_scale(word), z = (float)(word >> 16);
                unsigned dw = 0;
                if (!value)
                    dw = a.c.k_codes[(head * a.c.page_size + in_page + slot) * (D / 8) + q4_key_dword<D>(chunk)];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const unsigned q = value ? codes[wave][8 * chunk + i] >> (4 * (slot / 2 + 4 * (slot & 1))) & 15u
                                             : dw >> q4_shift(i) & 15u;
                    v[i] = (half_t)(s * ((float)q - z));
                }
            }
            *reinterpret_cast<half8 *>((value ? a.V : a.K) + ((int64_t)row * H + h) * D + 8 * chunk) = v;
        }
        q4_wave_fence();   // the next job's codes come after this one's reads
    }
}

// Workgroups for the heads of a granule.
static unsigned head_groups(int heads, int64_t granules)
{
    constexpr int64_t kWaves = 4096;
    const int64_t most = (heads + kCacheWaves - 1) / kCacheWaves, enough = (kWaves / kCacheWaves + granules - 1) / granules;
    return (unsigned)std::max<int64_t>(std::min(most, enough), 1);
}

template <int D, int GROUP>
static hipError_t launch_append(const Q4AppendArgs &a, hipStream_t s)
{
    const int jobs = 2 * a.c.heads + (a.Q ? a.q_heads : 0);
    const int64_t units = a.starts ? a.tokens / 8 + 2 * (int64_t)a.c.batch : a.c.batch;
    hipLaunchKernelGGL((q4_append_kernel<D, GROUP>), dim3((unsigned)units, head_groups(jobs, units)),
                       dim3(64 * kCacheWaves), 0, s, a);
    return hipGetLastError();
}

template <int D, int GROUP>
static hipError_t launch_read(const Q4ReadArgs &a, hipStream_t s)
{
    const int64_t units = a.tokens / 8 + 2 * (int64_t)a.c.batch;
    hipLaunchKernelGGL((q4_read_kernel<D, GROUP>),
                       dim3((unsigned)units, head_groups(2 * a.c.heads, units)),
                       dim3(64 * kCacheWaves), 0, s, a);
    return hipGetLastError();
}

#define GEMM_F16_Q4_FOR_CACHE(call)                                             \
    switch (a.c.head_dim * 1000 + a.c.group) {                                  \
    case 64032: return call<64, 32>(a, s);                                      \
    case 64064: return call<64, 64>(a, s);                                      \
    case 128032: return call<128, 32>(a, s);                                    \
    case 128064: return call<128, 64>(a, s);                                    \
    case 128128: return call<128, 128>(a, s);                                   \
    case 256032: return call<256, 32>(a, s);                                    \
    case 256064: return call<256, 64>(a, s);                                    \
    case 256128: return call<256, 128>(a, s);                                   \
    default: return hipErrorInvalidValue;                                       \
    }

hipError_t launch_q4_append(const Q4AppendArgs &a, hipStream_t s) { GEMM_F16_Q4_FOR_CACHE(launch_append) }

hipError_t launch_q4_read(const Q4ReadArgs &a, hipStream_t s) { GEMM_F16_Q4_FOR_CACHE(launch_read) }

} // namespace gemm_f16_impl
