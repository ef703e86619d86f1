// gemm_f16_q4_tile.hip -- the product with 4-bit weights, C = epi(alpha A W^T),
// LDS-staged tiles: for many rows of A, bound by the matrix cores, and for the
// few dozen rows where K is split.
//
// A workgroup's waves stand in WM rows: each owns 16 MB rows of A and 16 NW rows
// of W.  A stage holds 128 k: A's rows (256 bytes each), the workgroup's tiles of
// codes (1 KiB for each 16 rows of W) and their words, all moved straight from
// memory to LDS by buffer_load ... lds, STAGES - 1 stages ahead, with one barrier
// a stage.
//
// A's rows lie in LDS as 16 chunks of 16 bytes, chunk c of row r in place
// c ^ (r & 15): a fragment read takes one chunk of 16 rows, which then lie in
// 16 different 16-byte slots of the 256-byte bank window.  The lanes of a
// direct load fill LDS in order, so the permutation is made by the global
// address each lane loads.
//
// Scales.  The products of a group are summed in fp32 by the matrix cores and
// enter the total times the scale, as in the kernel for few rows: one fused
// multiply-add per output and group, so weights are used exactly, whatever the
// number of rows.  (A weight rounded to binary16 would need no sums of its own:
// 246, 251 and 273 us at 2048 x 8192 x 8192 with groups of 128, 64 and 32 where this
// took 271, 284 and 373 on the same machine; but s (q - z) has up to 15 bits, the rounding is as large as the
// result's own, and from 65520 on it is infinite.  Times in this file: captured
// calls one after the other, codes of random bits, inputs that no cache holds.)
//
// q4_128x256_s3 (8 waves): a wave of 128 rows by 32 of W unpacks each code once;
// for groups of 32, whose multiply-adds fill the vector unit, waves of 64 rows by
// 64 (two rows of waves, codes unpacked twice, half the reads of LDS) are faster
// (us at 2048 x 8192 x 8192 with groups of 128, 64, 32: 275, 284, 406 and 277, 299,
// 373).  Two waves on a SIMD, so that one's vector instructions run beside the
// other's matrix ones: 4 waves of 128 x 64 take 302, 398, 613.  Matrix instructions
// fill half of the SIMDs' cycles, vector ones (64 million) nearly as many; they
// overlap in part.  With weights of normal distribution, as in the timed case, groups
// of 128 take 241 (1140 TFLOP/s), and the dense kernel on binary16 weights 189.
//
// q4_64x128_s4 (8 waves): 64 x 8192 x 8192, group 64, in four parts of K, 21 us with
// the 4 of their sum, 18.5 alone under the profiler; whole 47, in two parts 30, in
// eight 25.  What bounds it is not found: vector instructions take 0.4 of the SIMDs'
// cycles and matrix ones 0.15, waves wait for 0.3, and neither 3, 5 or 6 stages, nor
// two workgroups on a CU (3 stages, 8 parts), nor half the reads of LDS (waves in
// two halves of k, two columns of blocks each), nor workgroups that start at
// different k change the time by more than 3 %.  Unsplit workgroups of the
// kernel for few rows take 23; 4 waves of 32 rows of W 24; 2 x 4 waves 22;
// codes 8 stages ahead by waves of their own 22; 64 x 256 in 8 parts 23.5.
#include "gemm_f16_q4_format.h"
#include "gemm_f16_tile.h"

namespace gemm_f16_impl {

typedef _Float16 half8_any __attribute__((ext_vector_type(8), aligned(2)));

template <int GROUP, int MB, int NW, int WM, int WAVES_, int STAGES_>
struct Q4Tile {
    static constexpr int WAVES = WAVES_, STAGES = STAGES_, GROUPS = 128 / GROUP, PER = GROUP / 32;
    static constexpr int BM = 16 * MB * WM, BN = 16 * NW * WAVES / WM, N_BLOCKS = NW * WAVES / WM;
    static constexpr int A_BYTES = BM * 256, CODE_BYTES = N_BLOCKS * 1024;
    static constexpr int A_LOADS = BM / 4 / WAVES, CODE_LOADS = N_BLOCKS / WAVES;   // of 1 KiB, for each wave
    static constexpr int WORD_LOADS = (N_BLOCKS * GROUPS / 4 + WAVES - 1) / WAVES;  // of 64 words
    static constexpr int STAGE_BYTES = A_BYTES + CODE_BYTES + WAVES * WORD_LOADS * 256;
    static constexpr int LOADS = A_LOADS + CODE_LOADS + WORD_LOADS;
    static constexpr int PITCH = BN + 8;                       // of the staged output, in halves
    static constexpr int LDS_BYTES = STAGES * STAGE_BYTES > BM * PITCH * 2 ? STAGES * STAGE_BYTES : BM * PITCH * 2;
    static_assert(BM / 4 % WAVES == 0 && N_BLOCKS % WAVES == 0, "whole loads for each wave");
    static_assert(LDS_BYTES <= 163840, "LDS of a CU");
};

// One stage's loads of a wave: 1 KiB pieces (of A: 4 rows; of the codes: a
// tile) and 256-byte pieces of the words, dealt out to the waves in turn.
template <class T>
struct Q4Loads {
    __amdgpu_buffer_rsrc_t a, codes, words;
    uint32_t a_off[T::A_LOADS];       // row and chunk of each load of A
    int chunk[T::A_LOADS];
    uint32_t code_off[T::CODE_LOADS], word_off[T::WORD_LOADS];
    int wave, lane, K, kb_end;

    __device__ __forceinline__ void init(const Q4Args &p, int m0, int nb0, int end)
    {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        K = p.K;
        kb_end = end;
        const int rows = min(p.M - m0, T::BM);
        a = make_rsrc(p.A + (int64_t)m0 * p.K, (uint32_t)rows * (uint32_t)p.K * 2u);
#pragma unroll
        for (int i = 0; i < T::A_LOADS; ++i) {
            const int row = 4 * (wave + T::WAVES * i) + lane / 16;
            chunk[i] = (lane & 15) ^ (row & 15);
            a_off[i] = (uint32_t)row * (uint32_t)p.K * 2u + (uint32_t)chunk[i] * 16u;
        }
        const int here = min(T::N_BLOCKS, p.n_blocks - nb0);   // past N: nothing is read
        const int64_t tile = (int64_t)nb0 * p.k_blocks;
        codes = make_rsrc(p.codes + tile * 256, (uint32_t)here * (uint32_t)p.k_blocks * 1024u);
        words = make_rsrc(p.words + tile * (16 * T::GROUPS), (uint32_t)here * (uint32_t)p.k_blocks * (64u * T::GROUPS));
#pragma unroll
        for (int i = 0; i < T::CODE_LOADS; ++i)
            code_off[i] = (uint32_t)(wave + T::WAVES * i) * (uint32_t)p.k_blocks * 1024u + (uint32_t)lane * 16u;
#pragma unroll
        for (int i = 0; i < T::WORD_LOADS; ++i) {
            const int w = 64 * (wave + T::WAVES * i) + lane, nb = w / (16 * T::GROUPS);
            word_off[i] = (nb < T::N_BLOCKS ? (uint32_t)nb * (uint32_t)p.k_blocks * (64u * T::GROUPS) : 0x80000000u) +
                          (uint32_t)(w % (16 * T::GROUPS)) * 4u;
        }
    }

    // block kb into the stage at `to`; blocks past the range bring zeros
    __device__ __forceinline__ void issue(int kb, unsigned char *to) const
    {
        const uint32_t gone = oob_unless(kb < kb_end);
#pragma unroll
        for (int i = 0; i < T::A_LOADS; ++i) {
            LDS_AS void *d = (LDS_AS void *)(to + (wave + T::WAVES * i) * 1024);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(a, d, 16, a_off[i] | gone | oob_unless(kb * 128 + chunk[i] * 8 < K),
                                                     (uint32_t)kb * 256u, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < T::CODE_LOADS; ++i) {
            LDS_AS void *d = (LDS_AS void *)(to + T::A_BYTES + (wave + T::WAVES * i) * 1024);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(codes, d, 16, code_off[i] | gone, (uint32_t)kb * 1024u, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < T::WORD_LOADS; ++i) {
            LDS_AS void *d = (LDS_AS void *)(to + T::A_BYTES + T::CODE_BYTES + (wave + T::WAVES * i) * 256);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(words, d, 4, word_off[i] | gone, (uint32_t)kb * (64u * T::GROUPS), 0, 0);
        }
    }

    // clear what the chunk that straddles the end of a row brought of the next row
    __device__ __forceinline__ void clear_tail(unsigned char *stage) const
    {
#pragma unroll 1
        for (int i = 0; i < T::A_LOADS; ++i) {
            const int piece = wave + T::WAVES * i, row = 4 * piece + lane / 16;
            if (((lane & 15) ^ (row & 15)) == K % 128 / 8) {
                unsigned char *c = stage + piece * 1024 + lane * 16;
                for (int e = K % 8; e < 8; e += 2)
                    *reinterpret_cast<uint32_t *>(c + 2 * e) = 0u;
            }
        }
    }
};

// TAIL: rows of A end inside a 16-byte chunk (K % 8 != 0).
template <class T, int MB, int NW, int WM, bool TAIL>
__device__ __forceinline__ void q4_tile(const Q4Args &p, unsigned char *lds)
{
    int tm, tn, split;
    tile_coords(blockIdx.x, gridDim.x, p.tiles_m, p.tiles_n, 4, tm, tn, split);
    const int m0 = tm * T::BM, nb0 = tn * T::N_BLOCKS;
    const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
    const int begin = split * p.split_blocks, end = min(p.k_blocks, begin + p.split_blocks);

    Q4Loads<T> in;
    in.init(p, m0, nb0, end);
    const int wave = in.wave / WM, wave_m = in.wave % WM;   // place along W's rows and along A's
    const q4_bits bits;

    float4v acc[MB][NW];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nw = 0; nw < NW; ++nw)
            acc[mb][nw] = float4v{0, 0, 0, 0};

#pragma unroll
    for (int s = 0; s < T::STAGES - 1; ++s)
        in.issue(begin + s, lds + s * T::STAGE_BYTES);

    // One stage: request block kb into `fill`, multiply the one in `from`.
    // (restrict: the stage being filled is not the one being read, so the
    // reads need not wait for the loads.)
    const auto step = [&](const unsigned char *__restrict__ from, unsigned char *__restrict__ fill, int kb)
                          __attribute__((always_inline)) {
        in.issue(kb, fill);
        const unsigned char *wc = from + T::A_BYTES + wave * (NW * 1024) + lane * 16;
        const uint32_t *ww = reinterpret_cast<const uint32_t *>(from + T::A_BYTES + T::CODE_BYTES) +
                             (wave * (NW * 16) + col) * T::GROUPS;
        uint4 codes[NW];
        unsigned word[NW][T::GROUPS];
#pragma unroll
        for (int nw = 0; nw < NW; ++nw) {
            codes[nw] = *reinterpret_cast<const uint4 *>(wc + nw * 1024);
#pragma unroll
            for (int q = 0; q < T::GROUPS; ++q)
                word[nw][q] = ww[nw * (16 * T::GROUPS) + q];
        }
#pragma unroll
        for (int q = 0; q < T::GROUPS; ++q) {
            half8 w[NW][T::PER];
            float s[NW];
#pragma unroll
            for (int nw = 0; nw < NW; ++nw) {
                const unsigned dw[4] = {codes[nw].x, codes[nw].y, codes[nw].z, codes[nw].w};
                const q4_zero zero(word[nw][q]);
#pragma unroll
                for (int j = 0; j < T::PER; ++j)
                    w[nw][j] = q4_codes(dw[q * T::PER + j], bits, zero);
                s[nw] = q4_scale(word[nw][q]);
            }
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
                float4v sum[NW];
#pragma unroll
                for (int j = 0; j < T::PER; ++j) {
                    const int chunk = 4 * (q * T::PER + j) + g;
                    const half8 a = *reinterpret_cast<const half8 *>(from + (wave_m * MB + mb) * 4096 + col * 256 +
                                                                     (chunk ^ col) * 16);
#pragma unroll
                    for (int nw = 0; nw < NW; ++nw)
                        sum[nw] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, w[nw][j], j == 0 ? float4v{0, 0, 0, 0} : sum[nw],
                                                                         0, 0, 0);
                }
#pragma unroll
                for (int nw = 0; nw < NW; ++nw)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[mb][nw][r] = __builtin_fmaf(s[nw], sum[nw][r], acc[mb][nw][r]);
            }
        }
    };

    int slot = 0;
    for (int kb = begin; kb < end; ++kb) {
        // this wave's loads of the stage have landed; and its reads of the
        // stage that is refilled next are done
        wait_vm_lgkm0<(T::STAGES - 2) * T::LOADS>();
        if constexpr (TAIL) {
            if (kb == p.k_blocks - 1) {
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
                in.clear_tail(lds + slot * T::STAGE_BYTES);
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            }
        }
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        const int fill = slot == 0 ? T::STAGES - 1 : slot - 1;
        step(lds + slot * T::STAGE_BYTES, lds + fill * T::STAGE_BYTES, kb + T::STAGES - 1);
        slot = slot + 1 == T::STAGES ? 0 : slot + 1;
    }
    wait_vmcnt<0>();   // the last requests' zeros land before LDS is used again or given back

    // lane (g, col) holds rows 16 mb + 4 g + r of the wave's, column col of each block
    const int rows = min(p.M - m0, T::BM), n0 = nb0 * 16, wave_n = wave * (16 * NW), row0 = wave_m * (16 * MB);
    if (p.W) {         // partial sums of a split, joined by the reduction kernel
        float *out = p.W + ((int64_t)split * p.M + m0) * p.N;
#pragma unroll
        for (int nw = 0; nw < NW; ++nw) {
            const int n = n0 + wave_n + nw * 16 + col;
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int m = row0 + 16 * mb + 4 * g + r;
                    if (m < rows && n < p.N)
                        out[(int64_t)m * p.N + n] = acc[mb][nw][r];
                }
        }
        return;
    }
    wait_lgkm0();
    __builtin_amdgcn_s_barrier();
    half_t *c = reinterpret_cast<half_t *>(lds);
#pragma unroll
    for (int nw = 0; nw < NW; ++nw)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float v = acc[mb][nw][r] * p.alpha;
                if (p.relu)
                    v = __builtin_fmaxf(v, 0.0f);
                c[(row0 + 16 * mb + 4 * g + r) * T::PITCH + wave_n + nw * 16 + col] = (half_t)v;
            }
    __syncthreads();
    constexpr int CHUNKS = T::BN / 8;
    for (int e = threadIdx.x; e < rows * CHUNKS; e += 64 * T::WAVES) {
        const int m = e / CHUNKS, n = e % CHUNKS * 8;
        const half8 v = *reinterpret_cast<const half8 *>(c + m * T::PITCH + n);
        half_t *to = p.C + (int64_t)(m0 + m) * p.N + n0 + n;
        if (n0 + n + 8 <= p.N) {
            __builtin_nontemporal_store(v, reinterpret_cast<half8_any *>(to));   // C streams out
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (n0 + n + i < p.N)
                    to[i] = v[i];
        }
    }
}

template <int GROUP, int MB, int NW, int WM, int WAVES, int STAGES, bool TAIL>
__global__ void __launch_bounds__(64 * WAVES) q4_tile_kernel(Q4Args p)
{
    typedef Q4Tile<GROUP, MB, NW, WM, WAVES, STAGES> T;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[T::LDS_BYTES];
    q4_tile<T, MB, NW, WM, TAIL>(p, lds);
}

template <int GROUP, bool TAIL>
static hipError_t launch_config(int config, const Q4Args &a, int64_t grid, hipStream_t s)
{
    const dim3 blocks((unsigned)grid), threads(512);
    constexpr int WM = GROUP == 32 ? 2 : 1;
    switch (config) {
    case 5: hipLaunchKernelGGL((q4_tile_kernel<GROUP, 4, 1, 1, 8, 4, TAIL>), blocks, threads, 0, s, a); break;
    case 6: hipLaunchKernelGGL((q4_tile_kernel<GROUP, 8 / WM, 2 * WM, WM, 8, 3, TAIL>), blocks, threads, 0, s, a); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <int GROUP>
static hipError_t launch_group(int config, const Q4Args &a, int64_t grid, hipStream_t s)
{
    return a.K % 8 != 0 ? launch_config<GROUP, true>(config, a, grid, s) : launch_config<GROUP, false>(config, a, grid, s);
}

hipError_t launch_q4_tile(int config, int group, const Q4Args &a, int64_t grid, hipStream_t s)
{
    return group == 32   ? launch_group<32>(config, a, grid, s)
           : group == 64 ? launch_group<64>(config, a, grid, s)
                         : launch_group<128>(config, a, grid, s);
}

} // namespace gemm_f16_impl
