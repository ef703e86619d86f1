// q4_extremes.cpp -- host-only driver of the 4-bit entry points at the ends of
// their arguments' ranges, built with AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_host_q4_extremes.py: validation of
// any sizes, strides and counts must not overflow, and what it lets through
// must describe buffers that an address space can hold.  The launchers are
// stubs; nothing is dereferenced.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include "gemm_f16_internal.h"
#include "gemm_f16_q4.h"
#include "gemm_f16_q4_format.h"

static int g_launches = 0, g_fails = 0, g_refused = 0;
#define CHECK(cond)                                                       \
    do {                                                                  \
        if (!(cond)) {                                                    \
            ++g_fails;                                                    \
            if (g_fails < 20)                                             \
                printf("failed: %s (line %d)\n", #cond, __LINE__);        \
        }                                                                 \
    } while (0)

static const double kSpace = 0x1p57;   // bytes

namespace gemm_f16_impl {
bool overlaps(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes)
{
    CHECK(a_bytes >= 0 && b_bytes >= 0 && (double)a_bytes <= kSpace && (double)b_bytes <= kSpace);
    if (a_bytes <= 0 || b_bytes <= 0)
        return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + (uintptr_t)b_bytes && b0 < a0 + (uintptr_t)a_bytes;
}
gemm_f16_status_t check_device(int *device)
{
    *device = 0;
    return GEMM_F16_SUCCESS;
}
static hipError_t launched()
{
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_q4(int, int, const Q4Args &, hipStream_t) { return launched(); }
hipError_t launch_q4_tile(int, int, const Q4Args &, int64_t, hipStream_t) { return launched(); }
hipError_t launch_q4_pack(const _Float16 *, _Float16 *, int64_t, int64_t, int64_t, hipStream_t) { return hipSuccess; }
hipError_t launch_q4_compress(const _Float16 *, uint32_t *, uint32_t *, int64_t, int64_t, int, bool, hipStream_t)
{
    return launched();
}
hipError_t launch_q4_expand(const uint32_t *, const uint32_t *, _Float16 *, int64_t, int64_t, int, hipStream_t)
{
    return launched();
}
hipError_t launch_reduce(const float *, _Float16 *, int64_t, int64_t, int, float, int, bool, hipStream_t) { return hipSuccess; }
static void fits(const Q4Pages &c)
{
    CHECK((double)c.pages * c.heads * c.page_size * c.head_dim / 2 <= kSpace);
    launched();
}
hipError_t launch_q4_append(const Q4AppendArgs &a, hipStream_t)
{
    fits(a.c);
    CHECK((double)a.tokens * a.k_stride * 2 <= kSpace && (double)a.tokens * a.v_stride * 2 <= kSpace);
    CHECK(!a.Q || (double)a.tokens * a.q_stride * 2 <= kSpace);
    CHECK(!a.cos || (double)a.positions * a.rotary * 2 <= kSpace);
    return hipSuccess;
}
hipError_t launch_q4_read(const Q4ReadArgs &a, hipStream_t)
{
    fits(a.c);
    return hipSuccess;
}
int64_t q4_attention_lds_bytes(int head_dim) { return 4 * kQ4AttentionWaves * (16 * (head_dim + 4) + 32); }
hipError_t launch_q4_attention(const Q4AttentionArgs &a, int64_t, hipStream_t)
{
    fits(a.c);
    CHECK((double)a.c.batch * a.q_stride * 2 <= kSpace);
    return hipSuccess;
}
} // namespace gemm_f16_impl

extern "C" gemm_f16_status_t gemm_f16_scaled(int64_t, int64_t, int64_t, const void *, int, const void *, int, void *, float, int, int,
                                             void *)
{
    return GEMM_F16_SUCCESS;
}

static uint64_t g_rng = 0x9E3779B97F4A7C15ull;
static uint64_t next()
{
    g_rng ^= g_rng << 13;
    g_rng ^= g_rng >> 7;
    g_rng ^= g_rng << 17;
    return g_rng;
}
// One of: a small number, the documented limit or near it, and the largest of the type.
static int64_t pick(int64_t limit, int64_t most)
{
    const int64_t from[] = {1, 8, 64, limit / 2, limit - 8, limit, limit < most ? limit + 1 : limit, most, most / 2 + 1, -1, INT64_MIN};
    const int64_t v = from[next() % (next() % 3 ? 6 : 11)];
    return v > most ? most : v;
}
static int small(int64_t v) { return v < INT32_MIN ? INT32_MIN : (int)v; }
static void *at(int i) { return (void *)((uint64_t)(i + 1) << 58); }

int main()
{
    for (int i = 0; i < 400000; ++i) {
        const int group = 32 << next() % 3;
        gemm_f16_status_t st;
        const int before = g_launches;
        switch (next() % 4) {
        case 0: {
            const int64_t M = pick(GEMM_F16_MAX_DIM, INT64_MAX), N = pick(GEMM_F16_MAX_N, INT64_MAX), K = pick(GEMM_F16_MAX_K, INT64_MAX);
            gemm_f16_plan_t plan;
            if (gemm_f16_plan_q4(M, N, K, group, nullptr, (int)(next() % 9) - 1, (int)(next() % 65), &plan) == GEMM_F16_SUCCESS)
                CHECK(plan.workspace_bytes >= 0 && plan.grid >= 0);
            (void)gemm_f16_q4_codes_bytes(N, K);
            (void)gemm_f16_q4_words_bytes(N, K, group);
            st = next() % 3 == 0   ? gemm_f16_q4_compress(N, K, group, 0, at(0), at(1), at(2), nullptr)
                 : next() % 2 == 0 ? gemm_f16_q4_expand(N, K, group, at(1), at(2), at(0), nullptr)
                                   : gemm_f16_q4(M, N, K, group, at(0), at(1), at(2), at(3), 1.0f, 0, -1, (int)(next() % 2), at(4),
                                                 INT64_MAX, nullptr);
            break;
        }
        default: {
            const gemm_f16_q4_cache_t c = {at(0), at(1), at(2), at(3), pick(GEMM_F16_Q4_MAX_PAGES, INT64_MAX),
                                           small(pick(GEMM_F16_Q4_MAX_HEADS, INT32_MAX)), small(pick(GEMM_F16_Q4_MAX_PAGE, INT32_MAX) & ~7LL),
                                           64 << next() % 3, group};
            const int64_t batch = pick(GEMM_F16_Q4_MAX_BATCH, INT64_MAX);
            const int64_t pages = c.page_size > 0 ? pick(GEMM_F16_Q4_MAX_LENGTH / c.page_size, INT64_MAX) : 1;
            const int64_t tokens = next() % 2 ? batch : pick(GEMM_F16_Q4_MAX_TOKENS, INT64_MAX);
            const int q_heads = next() % 2 ? c.heads : small(pick(GEMM_F16_Q4_MAX_HEADS, INT32_MAX));
            const int64_t stride = pick((int64_t)1 << 29, INT64_MAX) & ~7LL;
            const int kind = (int)(next() % 3);
            if (kind == 0)
                st = gemm_f16_q4_cache_append(&c, batch, tokens, pages, at(4), stride, at(5), pick((int64_t)1 << 29, INT64_MAX),
                                              (const int32_t *)at(6), (const int32_t *)at(7), (const int32_t *)at(8), at(9),
                                              pick((int64_t)1 << 29, INT64_MAX), at(10), q_heads, (const float *)at(11),
                                              (const float *)at(12), pick((int64_t)1 << 30, INT64_MAX), c.head_dim, 0, nullptr);
            else if (kind == 1)
                st = gemm_f16_q4_cache_read(&c, batch, tokens, pages, (const int32_t *)at(6), nullptr, (const int32_t *)at(8), at(4),
                                            at(5), nullptr);
            else
                st = gemm_f16_q4_attention(&c, batch, q_heads, pages, at(4), stride, (const int32_t *)at(6), (const int32_t *)at(7),
                                           0.1f, at(5), 1, pick(GEMM_F16_Q4_MAX_LENGTH, INT64_MAX), at(8), INT64_MAX, nullptr);
        }
        }
        CHECK(st >= GEMM_F16_SUCCESS && st <= GEMM_F16_ERROR_RUNTIME);
        g_refused += st != GEMM_F16_SUCCESS && g_launches == before;
    }
    printf("%d launches, %d refused, %d failed checks\n", g_launches, g_refused, g_fails);
    return g_fails != 0 || g_launches < 1000 || g_refused < 1000;
}
