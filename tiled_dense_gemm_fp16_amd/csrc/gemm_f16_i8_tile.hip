// gemm_f16_i8_tile.hip -- the product of two 8-bit matrices in LDS-staged tiles,
// dense or over the routed pairs of each expert.
//
// v_mfma_i32_16x16x64_i8 takes 16 bytes of each operand a lane and as many
// cycles as v_mfma_f32_16x16x32_f16 does, for twice the k.  Two neighbouring codes
// lie where one binary16 number would, so a tile is staged, swizzled and read
// as the binary16 tile of half the k is (Operand of gemm_f16_tile.h: 16-byte direct
// loads, conflict-free 16-byte fragment reads), and the balance of loads,
// LDS reads and matrix instructions is that tile's, at twice the rate.
//
// Sums are int32 and exact.  The product is computed transposed (W's fragment
// first), so a lane holds four neighbouring columns of one row of C.
//
// Tiles of 64 rows and more are computed by eight waves, two for each SIMD: their
// waits for loads overlap (four waves: 4096^3 58.8 us, eight 56.6; 64 tokens over 256
// experts 261, 241); 256 x 128 keeps four (1000 x 5000 x 4100 39.7 us, 41.7).  At
// 8192^3 (410 to 420 us, 2650 TOP/s; a library product reaches 2000) the matrix cores are busy
// 0.68 of the cycles and the clock falls to 1.8 GHz; smaller and colder products
// wait for memory (1000 x 5000 x 4100 busy 0.46, waves wait 0.32 of theirs; 2048 tokens
// over 64 experts 0.52, 0.44).  Slices of 64 bytes, of which twice as many are in
// flight, lose (4096^3 68 us; 2048 tokens 231, 194): half a cache line a row, and two
// barriers for one.
//
// 192 columns are there for products whose tiles of 256 leave CUs idle (1000 x 5000 x
// 4100, rows of 4224 bytes, 28 us in 216 workgroups, 32 in 160; 512 x 5000 x 8192 37, 40).
//
// Experts: a tile's rows of A are those of up to BM pairs of one expert, each
// fetched from where its row is (a direct load takes an address of its own
// for every 16 bytes anyway), and its rows of C go where their pairs are.
#include "gemm_f16_i8_device.h"

namespace gemm_f16_impl {

namespace {

// How a tile leaves: through LDS as 16-byte pieces of whole rows (C's rows
// 16-byte aligned), as a split's partial sums, or straight from the registers
// in 8- or 2-byte pieces.  Kernels of their own, as in gemm_f16_tile.h: a branch
// over them would move the accumulator out of the matrix unit's registers.
enum { kStaged, kPartial, kPieces };

// Words behind the stages, and all of a tile's LDS in halves.
template <int BM, int BN, int STAGES, int OUT, bool EXPERTS>
struct I8Lds {
    static constexpr int STAGE_HALVES = STAGES * (BM + BN) * (kI8BlockK / 2), OUT_HALVES = OUT == kStaged ? BM * BN : 0;
    static constexpr int TABLE_AT = STAGE_HALVES > OUT_HALVES ? STAGE_HALVES : OUT_HALVES;
    static constexpr int HALVES = TABLE_AT + 2 * ((EXPERTS ? 2 * BM : BM) + BN);
    static_assert(HALVES * 2 <= 163840, "LDS budget");
};

// A tile of C, or of a split's sums.  (lds is one array: with several, the compiler
// no longer sees that the loads into one stage leave the others alone, and waits
// for them before every read: 8192^3 425 us, 628 so.)
template <int BM, int BN, int WM, int WN, int STAGES, int OUT, bool EXPERTS>
__device__ __forceinline__ void i8_tile(const I8Args &p, half_t *lds, const I8Tile &t, int split)
{
    constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
    constexpr int BK = kI8BlockK / 2;                     // of a slice, as pairs of codes
    constexpr int TM = BM / WM / 16, TN = BN / WN / 16;   // 16 x 16 blocks of a wave
    using Op_a = Operand<true, BM, BK, THREADS, true, 8, true>;
    using Op_b = Operand<true, BN, BK, THREADS, true, 8, true>;
    constexpr int A_STAGE = Op_a::STAGE, B_STAGE = Op_b::STAGE, LOADS = Op_a::LOADS + Op_b::LOADS;
    half_t *const As = lds, *const Bs = lds + STAGES * A_STAGE;
    float *const column_scale = reinterpret_cast<float *>(lds + I8Lds<BM, BN, STAGES, OUT, EXPERTS>::TABLE_AT);
    float *const row_factor = column_scale + BN;
    int *const pairs = reinterpret_cast<int *>(row_factor + BM);   // experts

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm0 = (wave / WN) * (BM / WM), wn0 = (wave % WN) * (BN / WN);

    constexpr int MINE = (BM + THREADS - 1) / THREADS;   // rows tid, tid + THREADS, ... of the tile
    const int n0 = t.n0, rows = t.rows, m0 = EXPERTS ? 0 : t.first;
    int my_pair[MINE], my_row[MINE];
    const int8_t *W = p.W;
    const float *w_scales = p.w_scales;
    if constexpr (EXPERTS) {
#pragma unroll
        for (int i = 0; i < MINE; ++i)
            my_pair[i] = i8_pair(p, t, tid + i * THREADS);
        W += (int64_t)t.expert * p.N * p.w_pitch;
        w_scales += (int64_t)t.expert * p.N;
        if (t.expert >= p.experts) {   // pairs of no expert: zeros
#pragma unroll
            for (int i = 0; i < MINE; ++i)
                if (tid + i * THREADS < BM)
                    pairs[tid + i * THREADS] = my_pair[i];
            __syncthreads();
            const int most = min(BN, p.N - n0);
            for (int i = wave; i < rows; i += WAVES) {
                if (pairs[i] < 0)
                    continue;
                for (int n = lane; n < most; n += 64)
                    p.C[(int64_t)pairs[i] * p.N + n0 + n] = (half_t)0;
            }
            return;
        }
    }

    const int k_begin = split * p.k_split, k_end = min(p.K, k_begin + p.k_split);
    const int nk = (k_end - k_begin + kI8BlockK - 1) / kI8BlockK;

    Op_a opa;
    Op_b opb;
    opa.init(reinterpret_cast<const half_t *>(p.A), (int)(p.a_pitch / 2), m0, p.M, k_begin / 2, k_end / 2, tid, wave, lane);
    opb.init(reinterpret_cast<const half_t *>(W), (int)(p.w_pitch / 2), n0, p.N, k_begin / 2, k_end / 2, tid, wave, lane);
    int4v acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            acc[i][j] = int4v{0, 0, 0, 0};

    struct Frags {
        half8 x[TN], y[TM];
    };
    const auto load_frags = [&](Frags &f, const half_t *as, const half_t *bs, int ks) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
            f.y[i] = opa.frag16(as, wm0 + 16 * i, ks, lane);
#pragma unroll
        for (int j = 0; j < TN; ++j)
            f.x[j] = opb.frag16(bs, wn0 + 16 * j, ks, lane);
    };
    const auto mma = [&](const Frags &f) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int jj = 0; jj < TN; ++jj) {
                const int j = (i & 1) ? TN - 1 - jj : jj;   // neighbours share an operand
                acc[i][j] = i8_mfma(__builtin_bit_cast(int4v, f.x[j]), __builtin_bit_cast(int4v, f.y[i]), acc[i][j]);
            }
    };
    // Among the matrix instructions of one half step: the fragment reads of the
    // next one and the requests of a later slice, as in gemm_f16_tile.h.
    constexpr int MFMAS = TM * TN, READS = TM + TN;
    constexpr int READ_EVERY = MFMAS >= 2 * READS ? 2 : 1, READ_PER = (READS * READ_EVERY + MFMAS - 1) / MFMAS;
    const auto interleave = [&](int loads) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < MFMAS; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);          // one MFMA
#pragma unroll
            for (int r = 0; r < READ_PER; ++r)
                if (i % READ_EVERY == 0 && i / READ_EVERY * READ_PER + r < READS)
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // one LDS read
            if (i % 2 == 0 && i / 2 < loads)
                __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);      // one global load
        }
    };
    const auto issue = [&](int kt, half_t *a, half_t *b) __attribute__((always_inline)) {
        opa.issue(kt, a, wave);
        opb.issue(kt, b, wave);
    };
    // One slice, read from (rd_a, rd_b) while slice `next` is requested into
    // (wr_a, wr_b).  Fragments are read one 64-deep step ahead of their products:
    // f1 holds the second half of the slice before, if there is one.
    Frags f0, f1 = {};
    const auto step = [&](auto first, const half_t *__restrict__ rd_a, const half_t *__restrict__ rd_b, half_t *__restrict__ wr_a,
                          half_t *__restrict__ wr_b, int next) __attribute__((always_inline)) {
        issue(next, wr_a, wr_b);
        load_frags(f0, rd_a, rd_b, 0);
        if constexpr (!decltype(first)::value)
            mma(f1);
        interleave(LOADS);
        __builtin_amdgcn_sched_barrier(0);
        load_frags(f1, rd_a, rd_b, 1);
        mma(f0);
        interleave(0);
        __builtin_amdgcn_sched_barrier(0);
    };
    // Slice kt has landed for every wave, and every wave is done with the stage
    // that the next request fills.
    const auto ready = [&](int kt) __attribute__((always_inline)) {
        if (kt + STAGES - 2 < nk)
            wait_vm_lgkm0<(STAGES - 2) * LOADS>();
        else
            wait_vm_lgkm0<0>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    // The first requests.  (Over experts W's come before A's, whose rows have to pass
    // through LDS; which rows those are, and the expert, is known by now: the test for
    // pairs of none has waited for `order`.)
    if (nk > 0)
        opb.issue(0, Bs, wave);
    if constexpr (EXPERTS) {
        // where the tile's rows come from and go: places in A and C by way of LDS
#pragma unroll
        for (int i = 0; i < MINE; ++i) {
            const int at = tid + i * THREADS;
            my_row[i] = (int)((uint32_t)max(my_pair[i], 0) / (uint32_t)p.pairs_per_row);
            if (at < BM) {
                pairs[at] = my_pair[i];
                // (row_factor's place is free until then)
                reinterpret_cast<int *>(row_factor)[at] = my_pair[i] < 0 ? -1 : my_row[i];
            }
        }
        wait_lgkm0();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        opa.panel = make_rsrc(p.A, (uint32_t)p.M * (uint32_t)p.a_pitch);
#pragma unroll
        for (int i = 0; i < Op_a::DMA; ++i) {
            const int row = reinterpret_cast<const int *>(row_factor)[(wave * 64 + lane) / Op_a::CHUNKS + i * Op_a::ROW_STEP];
            const int col = Op_a::ALT_COLUMN && (i & 1) ? opa.kcol1 : opa.kcol0;
            opa.voff[i] = row < 0 ? 0x80000000u : (uint32_t)row * (uint32_t)p.a_pitch + (uint32_t)(2 * col);
        }
        wait_lgkm0();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    } else {
#pragma unroll
        for (int i = 0; i < MINE; ++i)
            my_row[i] = m0 + min(tid + i * THREADS, rows - 1);
    }
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s)
        if (s < nk) {
            opa.issue(s, As + s * A_STAGE, wave);
            if (s > 0)
                opb.issue(s, Bs + s * B_STAGE, wave);
        }
    // the factors of the tile's rows and columns, for the end (past the edges:
    // any, their products are not stored).  Loads arrive in order, so the waits for
    // these are waits for all slices requested above, too.
    if constexpr (OUT != kPartial) {
#pragma unroll
        for (int i = 0; i < MINE; ++i)
            if (tid + i * THREADS < BM)
                row_factor[tid + i * THREADS] = p.alpha * p.a_scales[my_row[i]];
        for (int i = tid; i < BN; i += THREADS)
            column_scale[i] = w_scales[min(n0 + i, p.N - 1)];
        asm volatile("" ::: "memory");   // written before the slices' barriers
    }
    constexpr int AHEAD = STAGES - 1;
    const auto stage = [&](auto first, int s, int kt) __attribute__((always_inline)) {
        const int w = (s + AHEAD) % STAGES;
        ready(kt);
        step(first, As + s * A_STAGE, Bs + s * B_STAGE, As + w * A_STAGE, Bs + w * B_STAGE, kt + AHEAD);
    };
    if (nk > 0)
        stage(std::integral_constant<bool, true>{}, 0, 0);
    // slices 1 ... in groups of STAGES, unrolled so that every stage is a constant
    for (int kt0 = 1; kt0 < nk; kt0 += STAGES) {
#pragma unroll
        for (int u = 0; u < STAGES; ++u)
            if (kt0 + u < nk)
                stage(std::integral_constant<bool, false>{}, (1 + u) % STAGES, kt0 + u);
    }
    mma(f1);
    wait_vmcnt<0>();   // the last requests land before the LDS is used again, or given up

    // Lane l holds, in block (i, j), columns wn0 + 16 j + 4 (l / 16) .. + 3 of row wm0 + 16 i + l % 16.
    const int row0 = wm0 + (lane & 15), col0 = wn0 + 4 * (lane >> 4);
    if constexpr (OUT == kPartial) {
        int *const to = p.partial + ((int64_t)split * p.M + m0) * p.N + n0;
        const __amdgpu_buffer_rsrc_t r = make_rsrc(to, ((uint32_t)rows * (uint32_t)p.N - (uint32_t)n0) * 4u);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int col = col0 + 16 * j;
                const uint32_t off = ((uint32_t)(row0 + 16 * i) * (uint32_t)p.N + (uint32_t)col) * 4u;
                if (p.N % 4 == 0) {
                    __builtin_amdgcn_raw_buffer_store_b128(acc[i][j], r, off | oob_unless(n0 + col < p.N), 0, 0);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        __builtin_amdgcn_raw_buffer_store_b32(acc[i][j][e], r, (off + 4u * e) | oob_unless(n0 + col + e < p.N), 0, 0);
                }
            }
    } else {
        if (nk == 0)
            __syncthreads();   // (the slices' barriers have ordered them otherwise)
        float factor[TM];
        float4v column[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i)
            factor[i] = row_factor[row0 + 16 * i];
#pragma unroll
        for (int j = 0; j < TN; ++j)
            column[j] = *reinterpret_cast<const float4v *>(column_scale + col0 + 16 * j);
        const auto out4 = [&](int i, int j, half_t (&h)[4]) __attribute__((always_inline)) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                h[e] = i8_out(acc[i][j][e], factor[i], column[j][e], p.relu);
        };
        // where row r of the tile goes, null for none
        const auto row_of_c = [&](int r) __attribute__((always_inline)) {
            if constexpr (EXPERTS)
                return pairs[r] < 0 ? (half_t *)nullptr : p.C + (int64_t)pairs[r] * p.N;
            else
                return r < rows ? p.C + (int64_t)(m0 + r) * p.N : (half_t *)nullptr;
        };
        if constexpr (OUT == kStaged) {
            // [BM][BN] in LDS, 8-byte units XOR-ed by row as in gemm_f16_tile.h
            // (within the largest power of two, up to 32, of which a row has a multiple)
            constexpr int UNITS = BN / 4, UMASK = (UNITS % 32 == 0 ? 32 : UNITS % 16 == 0 ? 16 : 8) - 1;
            wait_lgkm0();
            __builtin_amdgcn_s_barrier();   // every wave is done with the stages
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    half_t h[4];
                    out4(i, j, h);
                    const int r = row0 + 16 * i, u = (col0 + 16 * j) / 4;
                    *reinterpret_cast<half4 *>(lds + r * BN + 4 * (u ^ (r & UMASK))) = half4{h[0], h[1], h[2], h[3]};
                }
            wait_lgkm0();
            __builtin_amdgcn_s_barrier();
            constexpr int PIECES = BN / 8, EACH = (BM * PIECES + THREADS - 1) / THREADS;
#pragma unroll
            for (int q = 0; q < EACH; ++q) {
                const int id = tid + q * THREADS, r = id / PIECES, c = id % PIECES, sw = r & UMASK;
                if (BM * PIECES % THREADS != 0 && id >= BM * PIECES)
                    break;
                int4v v = *reinterpret_cast<const int4v *>(lds + r * BN + 4 * ((2 * c ^ sw) & ~1));
                if (sw & 1)
                    v = int4v{v[2], v[3], v[0], v[1]};
                half_t *const to = row_of_c(r);
                if (to && n0 + 8 * c < p.N)
                    __builtin_nontemporal_store(v, reinterpret_cast<int4v *>(to + n0 + 8 * c));
            }
        } else {
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                half_t *const to = row_of_c(row0 + 16 * i);
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const int n = n0 + col0 + 16 * j;
                    half_t h[4];
                    out4(i, j, h);
                    if (!to)
                        continue;
                    if (p.vec_c == 4) {
                        if (n < p.N)
                            __builtin_nontemporal_store(half4{h[0], h[1], h[2], h[3]}, reinterpret_cast<half4 *>(to + n));
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (n + e < p.N)
                                to[n + e] = h[e];
                    }
                }
            }
        }
    }
}

// CUT: the tiles of a last round that does not fill the card may be cut into
// quarters of BM / 2 by BN / 2, by as many waves with twice the stages, so that
// every CU has one.
template <int BM, int BN, int WM, int WN, int STAGES, int OUT, bool EXPERTS, bool CUT>
__global__ void __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(WM * WN / 4, WM * WN / 4)))
i8_tile_kernel(I8Args p)
{
    using Whole = I8Lds<BM, BN, STAGES, OUT, EXPERTS>;
    using Quarter = I8Lds<BM / 2, BN / 2, 2 * STAGES, OUT, EXPERTS>;
    constexpr int HALVES = CUT && Quarter::HALVES > Whole::HALVES ? Quarter::HALVES : Whole::HALVES;
    __shared__ __attribute__((aligned(1024))) half_t lds[HALVES];
    static_assert(sizeof(lds) == i8_lds_bytes(BM, BN, STAGES, EXPERTS), "as planned");
    I8Tile t;
    bool quarter = false;
    int split = 0;
    if constexpr (EXPERTS) {
        if (!i8_find_tile<BM, BN, CUT>(p, blockIdx.x, threadIdx.x & 63, t, quarter))
            return;
    } else {
        const int tiles = p.tiles_m * p.tiles_n;
        int id, tm, tn, part = 0;
        quarter = CUT && (int)blockIdx.x >= p.uncut;
        if (quarter) {   // the quarters of a tile to one XCD
            const int w = (int)blockIdx.x - p.uncut;
            id = p.uncut + w % 8 + w / 32 * 8;
            part = w / 8 % 4;
            if (id >= tiles)
                return;
        } else {
            id = i8_place(blockIdx.x, CUT ? p.uncut : (int)gridDim.x);
            split = id / tiles;
            id -= split * tiles;
        }
        i8_walk(id, p.tiles_m, p.tiles_n, tm, tn);
        t.first = tm * BM + part / 2 * (BM / 2);
        t.n0 = tn * BN + part % 2 * (BN / 2);
        t.rows = min(quarter ? BM / 2 : BM, p.M - t.first);
        t.expert = 0;
        if (t.rows <= 0 || t.n0 >= p.N)
            return;
    }
    if constexpr (CUT) {
        if (quarter) {
            i8_tile<BM / 2, BN / 2, WN, WM, 2 * STAGES, OUT, EXPERTS>(p, lds, t, split);
            return;
        }
    }
    i8_tile<BM, BN, WM, WN, STAGES, OUT, EXPERTS>(p, lds, t, split);
}

} // namespace

template <int BM, int BN, int WM, int WN, int STAGES, bool CUT = false>
static hipError_t launch_tile(const I8Args &a, int64_t grid, bool experts, hipStream_t s)
{
#define GEMM_F16_I8(OUT, EXPERTS, CUT_)                                                                                  \
    hipLaunchKernelGGL((i8_tile_kernel<BM, BN, WM, WN, STAGES, OUT, EXPERTS, CUT_>), dim3((unsigned)grid),              \
                       dim3(64 * WM * WN), 0, s, a)
    const bool cut = CUT && a.uncut < grid;
    if (experts && a.vec_c == 8)
        GEMM_F16_I8(kStaged, true, CUT);
    else if (experts)
        GEMM_F16_I8(kPieces, true, CUT);
    else if (a.partial)
        GEMM_F16_I8(kPartial, false, false);
    else if (a.vec_c == 8 && cut)
        GEMM_F16_I8(kStaged, false, CUT);
    else if (a.vec_c == 8)
        GEMM_F16_I8(kStaged, false, false);
    else if (cut)
        GEMM_F16_I8(kPieces, false, CUT);
    else
        GEMM_F16_I8(kPieces, false, false);
#undef GEMM_F16_I8
    return hipGetLastError();
}

hipError_t launch_i8_stream(const I8Args &a, int64_t grid, bool experts, hipStream_t s);

static hipError_t launch_config(int config, const I8Args &a, int64_t grid, bool experts, hipStream_t s)
{
    switch (config) {
    case 0: return launch_i8_stream(a, grid, experts, s);
    case 1: return launch_tile<32, 32, 2, 2, 8>(a, grid, experts, s);
    case 2: return launch_tile<32, 64, 1, 4, 6>(a, grid, experts, s);
    case 3: return launch_tile<64, 64, 2, 4, 6>(a, grid, experts, s);
    case 4: return launch_tile<64, 128, 2, 4, 4>(a, grid, experts, s);
    case 5: return launch_tile<64, 256, 1, 8, 3>(a, grid, experts, s);
    case 6: return launch_tile<128, 128, 2, 4, 4>(a, grid, experts, s);
    case 7: return launch_tile<128, 192, 2, 4, 3>(a, grid, experts, s);
    case 8: return launch_tile<128, 256, 2, 4, 3>(a, grid, experts, s);
    case 9: return launch_tile<256, 128, 2, 2, 3>(a, grid, experts, s);
    case 10: return launch_tile<256, 256, 4, 2, 2, true>(a, grid, experts, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_i8(int config, const I8Args &a, int64_t grid, hipStream_t s) { return launch_config(config, a, grid, false, s); }
hipError_t launch_i8_experts(int config, const I8Args &a, int64_t grid, hipStream_t s)
{
    return launch_config(config, a, grid, true, s);
}

} // namespace gemm_f16_impl
