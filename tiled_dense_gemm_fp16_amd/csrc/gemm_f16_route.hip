// gemm_f16_route.hip -- choice of experts from a token's logits, and the order
// of the chosen pairs by expert.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gemm_f16_i8_internal.h"
#include "gemm_f16_tile.h"

namespace gemm_f16_impl {

namespace {

typedef unsigned long long u64;

// What DPP control CTRL brings from another lane; lanes that it leaves out keep `old`.
template <int CTRL, int ROWS>
__device__ __forceinline__ unsigned dpp(unsigned old, unsigned x)
{
    return (unsigned)__builtin_amdgcn_update_dpp((int)old, (int)x, CTRL, ROWS, 0xf, false);
}
// Largest of a wave's 64 values: four steps inside the rows of 16 lanes, two across them.
__device__ __forceinline__ unsigned wave_max(unsigned x)
{
    x = max(x, dpp<0x111, 0xf>(0u, x));   // row_shr:1
    x = max(x, dpp<0x112, 0xf>(0u, x));   // row_shr:2
    x = max(x, dpp<0x114, 0xf>(0u, x));   // row_shr:4
    x = max(x, dpp<0x118, 0xf>(0u, x));   // row_shr:8
    x = max(x, dpp<0x142, 0xa>(0u, x));   // row_bcast:15
    x = max(x, dpp<0x143, 0xc>(0u, x));   // row_bcast:31
    return (unsigned)__builtin_amdgcn_readlane((int)x, 63);
}
__device__ __forceinline__ u64 lane_bits(u64 x, int lane)
{
    const unsigned lo = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)x, lane);
    const unsigned hi = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)(x >> 32), lane);
    return (u64)hi << 32 | lo;
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double x)   // 0 where there is no other lane
{
    const u64 b = __builtin_bit_cast(u64, x);
    return __builtin_bit_cast(double, (u64)dpp<CTRL, ROWS>(0u, (unsigned)(b >> 32)) << 32 | dpp<CTRL, ROWS>(0u, (unsigned)b));
}
__device__ __forceinline__ double wave_sum(double x)
{
    x += dpp<0x111, 0xf>(x);
    x += dpp<0x112, 0xf>(x);
    x += dpp<0x114, 0xf>(x);
    x += dpp<0x118, 0xf>(x);
    x += dpp<0x142, 0xa>(x);
    x += dpp<0x143, 0xc>(x);
    return __builtin_bit_cast(double, lane_bits(__builtin_bit_cast(u64, x), 63));
}

// Numbers as integers of the same order, all above 0, which stands for
// "closed" (+0 and -0 become one).
__device__ __forceinline__ u64 ordered(double x)
{
    const u64 b = __builtin_bit_cast(u64, x + 0.0);
    return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ u64 ordered(float x)
{
    const unsigned b = __builtin_bit_cast(unsigned, x + 0.0f);
    return (u64)(b >> 31 ? ~b : b | 1u << 31) << 32;
}

// The lane with the largest key, the lowest of equals; -1 where all are closed.
// High halves decide but for ties, which a second search resolves.
__device__ __forceinline__ int first_best(u64 key)
{
    const unsigned hi = (unsigned)(key >> 32), most = wave_max(hi);
    u64 at = __ballot(hi == most);
    if ((at & (at - 1)) != 0) {
        if (most == 0)   // (no number's high half)
            return -1;
        const unsigned lo = hi == most ? (unsigned)key : 0u, low = wave_max(lo);
        at = __ballot(hi == most && lo == low);
    }
    return __ffsll(at) - 1;
}

constexpr int kTokens = 4;   // waves of a workgroup, each with a token

// A wave takes a token; lane l holds the experts EACH l .. EACH l + EACH - 1, so
// that among equal keys the lowest lane has the lowest index.
// Keys are compared as integers, in 64 bits where scores enter them, so the
// choice is the definition's; without bias they are the logits themselves.
// A choice is a search over the wave in the vector unit's own lane moves
// (6 instructions where no two keys share their high half).  It is bound by the
// latency of these: each lane sorts its few keys first, so that a choice only
// moves up one lane's, and scores wait in LDS until the choices are made (64 tokens
// of 256 experts, 8 of them from 4 of 8 groups: 7.4 us; 8192 of 64, 6 of them: 6.4).
template <int EACH>
__global__ void __launch_bounds__(64 * kTokens) route_kernel(RouteArgs p)
{
    extern __shared__ double shared[];   // [kTokens][2][experts]: scores, and keys where there are groups
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t token = (int64_t)blockIdx.x * kTokens + wave;
    const int64_t from = (token < p.tokens ? token : p.tokens - 1) * p.stride;
    double *const scores = shared + 2 * wave * p.experts, *const keys = scores + p.experts;

    float x[EACH], bias[EACH];
    // (one branch around all loads, so that they are in flight together)
    if (p.half) {
#pragma unroll
        for (int i = 0; i < EACH; ++i)
            x[i] = (float)((const _Float16 *)p.logits)[from + min(lane * EACH + i, p.experts - 1)];
    } else {
#pragma unroll
        for (int i = 0; i < EACH; ++i)
            x[i] = ((const float *)p.logits)[from + min(lane * EACH + i, p.experts - 1)];
    }
#pragma unroll
    for (int i = 0; i < EACH; ++i)
        bias[i] = 0.0f;
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < EACH; ++i)
            bias[i] = p.bias[min(lane * EACH + i, p.experts - 1)];
    }
    float high = -INFINITY;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const bool open = lane * EACH + i < p.experts && x[i] > -INFINITY && bias[i] > -INFINITY;   // (neither is NaN)
        x[i] = open ? __builtin_fminf(x[i], 3.402823466e38f) : -INFINITY;
        high = __builtin_fmaxf(high, x[i]);
    }
    double score[EACH];
    if (!p.sigmoid) {
        const unsigned top = wave_max((unsigned)(ordered(high) >> 32));
        high = __builtin_bit_cast(float, top >> 31 ? top ^ 1u << 31 : ~top);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            score[i] = x[i] > -INFINITY ? exp((double)x[i] - (double)high) : 0.0;
            sum += score[i];
        }
        const double total = wave_sum(sum);
#pragma unroll
        for (int i = 0; i < EACH; ++i)
            score[i] = total > 0.0 ? score[i] / total : 0.0;
    } else {
#pragma unroll
        for (int i = 0; i < EACH; ++i)
            score[i] = x[i] > -INFINITY ? 1.0 / (1.0 + exp(-(double)x[i])) : 0.0;
    }
    u64 key[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int e = lane * EACH + i;
        const bool open = x[i] > -INFINITY;
        const double value = score[i] + (double)bias[i];
        key[i] = !open ? 0 : p.bias ? ordered(value) : ordered(x[i]);
        if (e < p.experts) {
            scores[e] = score[i];
            if (p.groups > 1)
                keys[e] = open ? value : -INFINITY;
        }
    }
    __syncthreads();

    if (p.groups > 1) {
        // two best keys of each group: a team of lanes for each, by way of LDS
        const int shift = p.team_shift, team = 1 << shift, size = p.group_size, g = lane >> shift;
        double a = -INFINITY, b = -INFINITY;   // the best and the next
        if (g < p.groups)
#pragma unroll 4
            for (int i = lane & (team - 1); i < size; i += team) {
                const double v = keys[g * size + i];
                b = v > a ? a : (v > b ? v : b);
                a = v > a ? v : a;
            }
        // (a team's lanes hold the same after each step, so a mirrored row swaps its halves)
        const auto merge = [&](double oa, double ob) {
            b = oa > a ? (a > ob ? a : ob) : (b > oa ? b : oa);
            a = oa > a ? oa : a;
        };
        if (team > 1)
            merge(dpp<0xb1, 0xf>(a), dpp<0xb1, 0xf>(b));     // quad_perm 1 0 3 2
        if (team > 2)
            merge(dpp<0x4e, 0xf>(a), dpp<0x4e, 0xf>(b));     // quad_perm 2 3 0 1
        if (team > 4)
            merge(dpp<0x141, 0xf>(a), dpp<0x141, 0xf>(b));   // row_half_mirror
        if (team > 8)
            merge(dpp<0x140, 0xf>(a), dpp<0x140, 0xf>(b));   // row_mirror
        for (int d = 16; d < team; d *= 2)
            merge(__shfl_xor(a, d), __shfl_xor(b, d));
        u64 best = 0;
        if ((lane & (team - 1)) == 0 && g < p.groups && a > -INFINITY)
            best = ordered(b > -INFINITY ? a + b : a);
        // a group stays if fewer than top_groups come before it
        int rank = 0;
        for (int other = 0; other < p.groups; ++other) {
            const u64 its = lane_bits(best, other << shift);
            rank += its > best || (its == best && other < g);
        }
        const u64 stay = __ballot(best != 0 && rank < p.top_groups);   // at the first lane of each team
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int e = lane * EACH + i;
            // e / size: the product is above the quotient by e / 2^22 at most, less than 1 / size
            if (e < p.experts && !(stay >> ((unsigned)e * p.group_magic >> 22 << shift) & 1))
                key[i] = 0;
        }
    }

    // the lane's own keys, the largest first, equals in the order of their indexes
    int which[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i)
        which[i] = i;
    constexpr bool SORTED = EACH <= 4;
    if constexpr (SORTED) {
#pragma unroll
        for (int n = EACH - 1; n > 0; --n)
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const bool swap = key[i + 1] > key[i];
                const u64 k = swap ? key[i] : key[i + 1];
                const int w = swap ? which[i] : which[i + 1];
                key[i] = swap ? key[i + 1] : key[i];
                which[i] = swap ? which[i + 1] : which[i];
                key[i + 1] = k;
                which[i + 1] = w;
            }
    }
    int my_id = -1;
    for (int j = 0; j < p.top_k; ++j) {
        u64 best = key[0];
        int its = which[0];
        if constexpr (!SORTED) {
#pragma unroll
            for (int i = 1; i < EACH; ++i)
                if (key[i] > best) {
                    best = key[i];
                    its = i;
                }
        }
        const int at = first_best(best);
        if (at < 0)
            break;
        const int e = at * EACH + __builtin_amdgcn_readlane(its, at);
        if (lane == j)
            my_id = e;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            if constexpr (SORTED) {
                if (lane == at) {
                    key[i] = i + 1 < EACH ? key[i + 1] : 0;
                    which[i] = i + 1 < EACH ? which[i + 1] : 0;
                }
            } else if (lane == at && its == i) {
                key[i] = 0;
            }
        }
    }
    double my_score = my_id >= 0 ? scores[my_id] : 0.0;
    if (p.renormalise) {
        double sum = my_score;
        for (int d = 1; d < p.top_k; d *= 2)   // (lanes from top_k on hold 0)
            sum += __shfl_xor(sum, d);
        my_score = sum > 0.0 ? my_score / sum : 0.0;
    }
    if (lane < p.top_k && token < p.tokens) {
        p.ids[token * p.top_k + lane] = my_id;
        p.weights[token * p.top_k + lane] = (float)((double)p.scale * my_score);
    }
}

// ---- the pairs by expert -----------------------------------------------------------
// A workgroup for each expert, and one for the pairs of none, finds the place
// of its first pair by counting the smaller ids itself, then writes its pairs:
// nothing passes between workgroups, and the order is that of the pairs.  Every
// workgroup reads all ids, from the L2s.  Where CUs are left over, several share an
// expert, each writing the pairs of one part of the ids (it counts the equal ids
// of the parts before it, too).
//
// It is bound by the instructions for each id, so a wave keeps of its part's ids
// only one bit each, ROUNDS times 4 a lane, and the ranks of three rounds
// (256 ids each, at most 256 equal) pass through one sum over the wave: 512 pairs
// over 256 experts 2.9 us, 49152 over 64 experts 8.8.
__device__ __forceinline__ unsigned wave_upto(unsigned x)   // inclusive sums
{
    x += dpp<0x111, 0xf>(0u, x);
    x += dpp<0x112, 0xf>(0u, x);
    x += dpp<0x114, 0xf>(0u, x);
    x += dpp<0x118, 0xf>(0u, x);
    x += dpp<0x142, 0xa>(0u, x);
    x += dpp<0x143, 0xc>(0u, x);
    return x;
}

template <int WAVES, int ROUNDS>
__global__ void __launch_bounds__(64 * WAVES) expert_order_kernel(const int32_t *__restrict__ ids, int32_t *__restrict__ order,
                                                                  int32_t *__restrict__ starts, int pairs, int experts, int part)
{
    static_assert(ROUNDS % 3 == 0 && ROUNDS <= 8 * 2 * 3, "whole sums");
    constexpr int WORDS = (ROUNDS + 5) / 6;   // 6 rounds' bits in a word
    __shared__ int below[WAVES], earlier[WAVES], equal[WAVES];
    const int expert = blockIdx.x, lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool none = expert == experts;
    const __amdgpu_buffer_rsrc_t all = make_rsrc(ids, (uint32_t)pairs * 4u);   // past the end: zeros
    const auto load = [&](int at) {
        return __builtin_bit_cast(int4v, __builtin_amdgcn_raw_buffer_load_b128(all, (uint32_t)(at + 4 * lane) * 4u, 0, 0));
    };
    const auto is_less = [&](int id) { return (unsigned)id < (unsigned)expert; };
    const auto is_mine = [&](int id) { return none ? (unsigned)id >= (unsigned)experts : id == expert; };

    // the other parts, 256 ids at a time (a part is a multiple of that)
    const int first = min((int)blockIdx.y * part, pairs), last = min(first + part, pairs);
    int less = 0, before = 0;
    if (gridDim.y > 1) {
        constexpr int AT_ONCE = 4;
        for (int at0 = wave * AT_ONCE * 256; at0 < pairs; at0 += WAVES * AT_ONCE * 256) {
            int4v v[AT_ONCE];
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i)
                v[i] = load(at0 + 256 * i);
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                const int at = at0 + 256 * i;
                if (at >= pairs || (at >= first && at < last))
                    continue;
                if (at < first) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        less += is_less(v[i][r]);
                        before += is_mine(v[i][r]);
                    }
                } else {
                    const bool whole = at + 256 <= pairs;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        less += is_less(v[i][r]) && (whole || at + 4 * lane + r < pairs);
                }
            }
        }
    }

    // this part: a run of `rounds` rounds for each wave, ROUNDS of them at a time
    const int rounds = (last - first + 256 * WAVES - 1) / (256 * WAVES);
    const int begin = first + wave * rounds * 256;
    unsigned bits[WORDS];
    const auto look = [&](int r0) __attribute__((always_inline)) {
        int4v v[ROUNDS];
#pragma unroll
        for (int h = 0; h < ROUNDS; ++h)
            if (r0 + h < rounds)
                v[h] = load(begin + (r0 + h) * 256);
        int smaller = 0;
#pragma unroll
        for (int w = 0; w < WORDS; ++w)
            bits[w] = 0;
#pragma unroll
        for (int h = 0; h < ROUNDS; ++h) {
            if (r0 + h >= rounds)
                continue;
            const int at = begin + (r0 + h) * 256;
            unsigned four = 0;
            if (at + 256 <= last) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    smaller += is_less(v[h][r]);
                    four |= is_mine(v[h][r]) ? 1u << r : 0u;
                }
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool in = at + 4 * lane + r < last;
                    smaller += in && is_less(v[h][r]);
                    four |= in && is_mine(v[h][r]) ? 1u << r : 0u;
                }
            }
            bits[h / 6] |= four << (4 * (h % 6));
        }
        return smaller;
    };
    int same = 0;
    for (int r0 = 0; r0 < rounds; r0 += ROUNDS) {
        less += look(r0);
#pragma unroll
        for (int w = 0; w < WORDS; ++w)
            same += __popc(bits[w]);
    }
    less = (int)wave_upto((unsigned)less);
    before = (int)wave_upto((unsigned)before);
    same = (int)wave_upto((unsigned)same);
    if (lane == 63) {
        below[wave] = less;
        earlier[wave] = before;
        equal[wave] = same;
    }
    __syncthreads();
    int place = 0;
    for (int w = 0; w < WAVES; ++w)
        place += below[w];
    if (threadIdx.x == 0 && blockIdx.y == 0)
        starts[expert] = place;
    for (int w = 0; w < WAVES; ++w)
        place += earlier[w];
    for (int w = 0; w < wave; ++w)
        place += equal[w];
    if (__builtin_amdgcn_readlane(same, 63) == 0)
        return;
    for (int r0 = 0; r0 < rounds; r0 += ROUNDS) {
        if (rounds > ROUNDS)
            look(r0);
#pragma unroll
        for (int h0 = 0; h0 < ROUNDS; h0 += 3) {
            unsigned mine = 0;   // of three rounds, in 10 bits each
#pragma unroll
            for (int i = 0; i < 3; ++i)
                mine |= (unsigned)__popc(bits[(h0 + i) / 6] >> (4 * ((h0 + i) % 6)) & 15u) << (10 * i);
            const unsigned upto = wave_upto(mine), total = (unsigned)__builtin_amdgcn_readlane((int)upto, 63);
            if (total == 0)
                continue;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                unsigned four = bits[(h0 + i) / 6] >> (4 * ((h0 + i) % 6)) & 15u;
                int to = place + (int)((upto - mine) >> (10 * i) & 1023u);
                const int at = begin + (r0 + h0 + i) * 256 + 4 * lane;
                while (four) {
                    order[to++] = at + __ffs(four) - 1;
                    four &= four - 1;
                }
                place += (int)(total >> (10 * i) & 1023u);
            }
        }
    }
}

} // namespace

hipError_t launch_route(const RouteArgs &args, hipStream_t s)
{
    RouteArgs a = args;
    a.group_size = a.experts / a.groups;
    a.group_magic = (1u << 22) / (unsigned)a.group_size + 1;
    a.team_shift = 6;
    while (a.groups << a.team_shift > 64)
        --a.team_shift;
    const dim3 grid((unsigned)((a.tokens + kTokens - 1) / kTokens));
    const unsigned lds = (unsigned)(kTokens * 2 * a.experts * sizeof(double));
#define GEMM_F16_ROUTE(EACH) hipLaunchKernelGGL(route_kernel<EACH>, grid, dim3(64 * kTokens), lds, s, a)
    if (a.experts <= 64)
        GEMM_F16_ROUTE(1);
    else if (a.experts <= 128)
        GEMM_F16_ROUTE(2);
    else if (a.experts <= 256)
        GEMM_F16_ROUTE(4);
    else if (a.experts <= 512)
        GEMM_F16_ROUTE(8);
    else
        GEMM_F16_ROUTE(16);
#undef GEMM_F16_ROUTE
    return hipGetLastError();
}

hipError_t launch_expert_order(const int32_t *ids, int32_t *order, int32_t *starts, int pairs, int experts, hipStream_t s)
{
    if (pairs <= 4 * 3 * 256) {
        hipLaunchKernelGGL((expert_order_kernel<4, 3>), dim3((unsigned)(experts + 1)), dim3(256), 0, s, ids, order, starts, pairs,
                           experts, pairs);
    } else {
        // parts of 4096 ids and more, as many as leave each workgroup a CU
        const int parts = std::max(1, std::min(256 / (experts + 1), pairs / 4096));
        const int part = ((pairs + parts - 1) / parts + 255) / 256 * 256;
        hipLaunchKernelGGL((expert_order_kernel<16, 12>), dim3((unsigned)(experts + 1), (unsigned)parts), dim3(1024), 0, s, ids, order,
                           starts, pairs, experts, part);
    }
    return hipGetLastError();
}

} // namespace gemm_f16_impl
