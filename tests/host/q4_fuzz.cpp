// q4_fuzz.cpp -- host-only driver for the validation and planning of the
// 4-bit entry points, built with AddressSanitizer and UndefinedBehaviorSanitizer
// by tests/test_host_q4_sanitized.py.  The kernel launchers are replaced by
// stubs that check what reaches them: sizes within what the kernels assume,
// split ranges that cover K without an empty one, a page division that agrees
// with the plain one.  Pointers are stand-ins that nothing dereferences.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "gemm_f16_internal.h"
#include "gemm_f16_q4.h"
#include "gemm_f16_q4_format.h"

static int g_launches = 0, g_fails = 0;
#define CHECK(cond)                                                       \
    do {                                                                  \
        if (!(cond)) {                                                    \
            ++g_fails;                                                    \
            if (g_fails < 20)                                             \
                printf("failed: %s (line %d)\n", #cond, __LINE__);        \
        }                                                                 \
    } while (0)

namespace gemm_f16_impl {
bool overlaps(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes)
{
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
static void check_product(const Q4Args &a, int group)
{
    ++g_launches;
    CHECK(a.M > 0 && a.N > 0 && a.K >= 0 && a.C && (a.K == 0 || (a.A && a.codes && a.words)));
    CHECK(group == 32 || group == 64 || group == 128);
    CHECK(a.n_blocks == (a.N + 15) / 16 && a.k_blocks == (a.K + 127) / 128);
    CHECK(a.splits >= 1 && a.splits <= GEMM_F16_MAX_SPLITS && (a.splits > 1) == (a.W != nullptr));
    CHECK((int64_t)a.splits * a.split_blocks >= a.k_blocks);
    CHECK(a.k_blocks == 0 || (int64_t)(a.splits - 1) * a.split_blocks < a.k_blocks);
    CHECK(a.rows == a.M && a.row0 == 0);
}
hipError_t launch_q4(int config, int group, const Q4Args &a, hipStream_t)
{
    CHECK(config >= 0 && config < kQ4Expanded && kQ4Configs[config].stages == 0);
    CHECK((int64_t)a.tiles_m * 16 * kQ4Configs[config].m_blocks >= a.M);
    CHECK((int64_t)a.tiles_n * kQ4Configs[config].n_blocks >= a.n_blocks);
    check_product(a, group);
    return hipSuccess;
}
hipError_t launch_q4_tile(int config, int group, const Q4Args &a, int64_t grid, hipStream_t)
{
    CHECK(config >= 0 && config < kNumQ4Configs && kQ4Configs[config].stages > 0);
    CHECK((uintptr_t)a.A % 4 == 0 && a.K % 2 == 0);
    CHECK(grid == (int64_t)a.tiles_m * a.tiles_n * a.splits && grid * 64 * kQ4Configs[config].waves <= 0xffffffff);
    check_product(a, group);
    return hipSuccess;
}
static int g_packs = 0;
hipError_t launch_q4_pack(const _Float16 *A, _Float16 *to, int64_t M, int64_t K, int64_t pitch, hipStream_t)
{
    ++g_packs;
    CHECK(A && to && (uintptr_t)to % 16 == 0 && M > 0 && K > 0 && pitch >= K && pitch < K + 8 && pitch % 8 == 0);
    return hipSuccess;
}
hipError_t launch_q4_compress(const _Float16 *W, uint32_t *codes, uint32_t *words, int64_t N, int64_t K, int group, bool,
                              hipStream_t)
{
    ++g_launches;
    CHECK(W && codes && words && N > 0 && K > 0 && (group == 32 || group == 64 || group == 128));
    return hipSuccess;
}
hipError_t launch_q4_expand(const uint32_t *codes, const uint32_t *words, _Float16 *W, int64_t N, int64_t K, int group,
                            hipStream_t s)
{
    return launch_q4_compress(W, const_cast<uint32_t *>(codes), const_cast<uint32_t *>(words), N, K, group, false, s);
}
hipError_t launch_reduce(const float *W, _Float16 *, int64_t M, int64_t N, int splits, float, int, bool, hipStream_t)
{
    CHECK(W && M > 0 && N > 0 && splits > 1);
    return hipSuccess;
}
static void check_pages(const Q4Pages &c)
{
    ++g_launches;
    CHECK(c.page_size >= 8 && c.page_size % 8 == 0 && c.heads > 0 && c.batch > 0);
    CHECK(c.max_pages == 0 || c.table);
    const uint32_t last = (uint32_t)1 << 31;
    for (uint32_t t : {0u, 1u, (uint32_t)c.page_size - 1, (uint32_t)c.page_size, (uint32_t)c.page_size + 1, last - 1,
                       last / 3, (uint32_t)c.page_size * 1000u + 7u})
        if (t < last)
            CHECK((uint32_t)(((uint64_t)t * c.page_magic >> 32) >> c.page_shift) == t / (uint32_t)c.page_size);
}
hipError_t launch_q4_append(const Q4AppendArgs &a, hipStream_t)
{
    check_pages(a.c);
    CHECK(a.K && a.V && a.lengths && a.tokens > 0 && (a.starts || a.tokens == a.c.batch));
    CHECK(!a.Q == !a.Q_out && (!a.Q || a.q_heads > 0) && !a.cos == !a.sin && a.rotary % 16 == 0 && a.rotary <= a.c.head_dim);
    CHECK(a.c.pages == 0 || a.c.k_codes);
    CHECK(((int64_t)a.tokens / 8 + 2 * (int64_t)a.c.batch) * 256 <= 0xffffffff);
    return hipSuccess;
}
hipError_t launch_q4_read(const Q4ReadArgs &a, hipStream_t)
{
    check_pages(a.c);
    CHECK(a.K && a.V && a.starts && a.tokens > 0);
    return hipSuccess;
}
int64_t q4_attention_lds_bytes(int head_dim) { return 4 * kQ4AttentionWaves * (16 * (head_dim + 4) + 32); }
hipError_t launch_q4_attention(const Q4AttentionArgs &a, int64_t grid, hipStream_t)
{
    check_pages(a.c);
    CHECK(a.Q && a.out && a.lengths && a.ratio * a.c.heads == a.q_heads && a.row_tiles * 16 >= a.ratio);
    CHECK(grid == (int64_t)a.c.batch * a.c.heads * a.row_tiles * a.splits && grid * 256 <= 0xffffffff);
    CHECK(a.step == 32 || (a.step == 64 && a.ratio <= 8) || (a.step == 128 && a.ratio <= 4 && a.c.head_dim < 256));
    CHECK((a.splits > 1) == (a.parts != nullptr) && (a.c.pages > 0 || a.c.max_pages == 0));
    return hipSuccess;
}
} // namespace gemm_f16_impl

extern "C" gemm_f16_status_t gemm_f16_scaled(int64_t M, int64_t N, int64_t K, const void *A, int trans_a, const void *B, int trans_b,
                                             void *C, float, int epilogue, int config, void *)
{
    CHECK(M > 0 && N > 0 && K >= 0 && C && !trans_a && trans_b == 1 && config == GEMM_F16_CONFIG_AUTO);
    CHECK(K == 0 || (A && B && (uintptr_t)B % 16 == 0));
    CHECK(epilogue == GEMM_F16_EPILOGUE_NONE || epilogue == GEMM_F16_EPILOGUE_RELU);
    g_launches += K == 0;   // (with K > 0 the expansion before it is counted)
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
static int64_t pick(int64_t most)
{
    static const int64_t edges[] = {0, 1, 2, 7, 8, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 256, 4100, 8192, 28672,
                                    (int64_t)1 << 20, ((int64_t)1 << 22) + 1, (int64_t)1 << 26, (int64_t)1 << 31, -1};
    return next() % 8 == 0 ? edges[next() % (sizeof(edges) / sizeof(edges[0]))] : (int64_t)(next() % (uint64_t)most);
}
static void *at(int i)
{
    const uint64_t odd[] = {0, 0, 0, 0, 0, 0, 2, 4, 8, 1};
    return next() % 40 == 0 ? nullptr : (void *)(((uint64_t)(i + 1) << 48) + odd[next() % 10]);
}
static int group() { return next() % 12 ? 32 << next() % 3 : (int)(next() % 200); }

int main()
{
    int ok = 0;
    for (int i = 0; i < 400000; ++i) {
        const int before = g_launches;
        gemm_f16_status_t st;
        bool nothing = false;
        const int kind = (int)(next() % 5);
        if (kind == 0) {
            const int64_t M = next() % 6 ? pick(600) : 2000 + pick(600), N = pick(5000), K = pick(9000);
            const int gr = group(), config = (int)(next() % 10) - 1, splits = next() % 3 ? 0 : (int)(next() % 70) - 1;
            gemm_f16_plan_t plan;
            void *A = at(0), *ws = next() % 2 ? at(4) : nullptr;
            st = gemm_f16_q4(M, N, K, gr, A, at(1), at(2), at(3), 0.5f, (int)(next() % 3), config, splits, ws,
                             ws ? (int64_t)(next() % ((uint64_t)1 << 40)) : 0, nullptr);
            if (st == GEMM_F16_SUCCESS) {
                CHECK(gemm_f16_plan_q4(M, N, K, gr, A, config, splits, &plan) == GEMM_F16_SUCCESS);
                CHECK(plan.splits >= 1 && plan.lds_bytes <= 163840);
            }
            nothing = M == 0 || N == 0;
        } else if (kind == 1) {
            const int64_t N = pick(5000), K = pick(9000);
            st = next() % 2 ? gemm_f16_q4_compress(N, K, group(), (int)(next() % 3), at(0), at(1), at(2), nullptr)
                            : gemm_f16_q4_expand(N, K, group(), at(1), at(2), at(0), nullptr);
            nothing = N == 0 || K == 0;
        } else {
            gemm_f16_q4_cache_t c = {at(5), at(6), at(7), at(8), pick(100000), (int32_t)pick(70), (int32_t)(8 * pick(70)),
                                     next() % 10 ? 64 << next() % 3 : (int32_t)pick(300), group()};
            const int64_t batch = pick(300), tokens = next() % 3 ? pick(5000) : batch, pages = pick(500);
            const int64_t width = (int64_t)c.heads * c.head_dim, q_heads = next() % 5 ? c.heads * (int64_t)(next() % 20) : pick(100);
            nothing = batch == 0 || tokens == 0;
            if (kind == 2) {
                void *q = next() % 2 ? at(4) : nullptr;
                const float *cos = next() % 2 ? (const float *)at(11) : nullptr;
                st = gemm_f16_q4_cache_append(next() % 50 ? &c : nullptr, batch, tokens, pages, at(0), width + pick(100), at(1),
                                              width + pick(100), (const int32_t *)at(2), (const int32_t *)at(3),
                                              next() % 2 ? (const int32_t *)at(9) : nullptr, q, q_heads * c.head_dim + pick(100),
                                              q ? at(10) : nullptr, (int)q_heads, cos, cos ? (const float *)at(12) : nullptr,
                                              pick(100000), cos ? 16 * (int)(next() % 18) : 0, (int)(next() % 2), nullptr);
            } else if (kind == 3) {
                st = gemm_f16_q4_cache_read(&c, batch, tokens, pages, (const int32_t *)at(2),
                                            next() % 2 ? (const int32_t *)at(3) : nullptr, (const int32_t *)at(9), at(0), at(1),
                                            nullptr);
            } else {
                void *ws = next() % 2 ? at(4) : nullptr;
                st = gemm_f16_q4_attention(&c, batch, (int)q_heads, pages, at(0), q_heads * c.head_dim + 8 * pick(30),
                                           (const int32_t *)at(2), (const int32_t *)at(3), 0.1f, at(1),
                                           next() % 2 ? 0 : (int)(next() % 300) - 10, pick(100000), ws,
                                           ws ? (int64_t)(next() % ((uint64_t)1 << 40)) : 0, nullptr);
                nothing = batch == 0;
            }
        }
        CHECK(st >= GEMM_F16_SUCCESS && st <= GEMM_F16_ERROR_RUNTIME);
        CHECK(g_launches - before == (st == GEMM_F16_SUCCESS && !nothing ? 1 : 0));
        ok += st == GEMM_F16_SUCCESS;
    }
    printf("%d calls accepted, %d launches, %d failed checks\n", ok, g_launches, g_fails);
    return g_fails != 0;
}
