// Host-side checks of the sampling, truncated verification and paged cache
// calls under AddressSanitizer and UndefinedBehaviorSanitizer (test
// infrastructure, CPU only): sv_sample_api.cpp and sv_cache_api.cpp linked
// against stub launchers.  A call is refused without reaching a stub, or
// reaches it with arguments that a kernel could use: the stubs check the plan.
#include <cstdio>
#include <limits>

#include "libspecverify.h"
#include "sv_launch.h"
#include "sv_serve.h"

static int g_launches = 0, g_failures = 0;

#define EXPECT(cond)                                                       \
    do {                                                                   \
        if (!(cond)) {                                                     \
            std::fprintf(stderr, "FAILED line %d: %s\n", __LINE__, #cond); \
            ++g_failures;                                                  \
        }                                                                  \
    } while (0)

namespace sv {
sv_status finish_launch(hipError_t e, hipStream_t) { return e == hipSuccess ? SV_OK : SV_ERR_LAUNCH; }
hipError_t launch_sample(const SampleArgs& a, hipStream_t) {
    ++g_launches;
    EXPECT(a.n_rows > 0 && a.vocab > 0);
    return hipErrorNotSupported;
}
hipError_t launch_verify_truncated(const VerifyTruncatedArgs& a, hipStream_t) {
    ++g_launches;
    EXPECT(a.laws != nullptr && a.n_req > 0);
    return hipErrorNotSupported;
}
hipError_t launch_cache_append(const AppendArgs& a, hipStream_t) {
    ++g_launches;
    EXPECT((int64_t)a.n_rows * 2 * a.cache.n_kv_heads * (a.cache.head_dim / 8) < ((int64_t)1 << 32));
    return hipErrorNotSupported;
}
hipError_t launch_cache_attend(const AttendArgs& a, hipStream_t) {
    ++g_launches;
    const int64_t grid =
        (int64_t)a.n_req * a.cache.n_kv_heads * a.slot_blocks * a.parts;
    EXPECT(grid > 0 && grid * 256 < ((int64_t)1 << 32));
    EXPECT(a.slot_blocks * 16 * a.slot_tiles >= (a.k_max + 1) * a.group);
    EXPECT(a.parts >= 1 && a.parts <= 128 && a.part_min % 128 == 0 && a.part_min > 0);
    EXPECT(a.parts == 1 || (a.part_out != nullptr && a.part_ml != nullptr));
    // the parts cover any length the table holds
    const int64_t capacity = (int64_t)a.max_pages * a.cache.page_size;
    for (int64_t len : {(int64_t)1, capacity / 2, capacity})
        if (len > 0 && len < (1 << 30))
            EXPECT((int64_t)part_len((int)len, a.parts, a.part_min) * a.parts >= len);
    return hipErrorNotSupported;
}
}  // namespace sv

int main() {
    alignas(16) static float fake[64];
    void* F = fake;
    const float* cf = fake;
    float* mf = fake;
    int32_t* mi = reinterpret_cast<int32_t*>(fake);
    const int32_t* ci = mi;
    const sv_sampling law{cf, ci, cf, nullptr};

    int before = g_launches;
    EXPECT(sv_sample(F, 10, 2, (sv_dtype)7, 10, &law, cf, mi, mf, mi, mi, nullptr) == SV_ERR_DTYPE);
    EXPECT(sv_sample(F, 9, 2, SV_F32, 10, &law, cf, mi, mf, mi, mi, nullptr) == SV_ERR_SHAPE);
    EXPECT(sv_sample(F, std::numeric_limits<int64_t>::max(), 4, SV_F32, 10, nullptr, cf, mi, mf, mi,
                     mi, nullptr) == SV_ERR_SHAPE);
    EXPECT(sv_sample(nullptr, 10, 2, SV_F32, 10, &law, cf, mi, mf, mi, mi, nullptr) == SV_ERR_NULL);
    EXPECT(g_launches == before);
    EXPECT(sv_sample(F, 10, 2, SV_F32, 10, &law, cf, mi, nullptr, nullptr, nullptr, nullptr) ==
           SV_ERR_LAUNCH);
    EXPECT(sv_sample(F, 10, 2, SV_BF16, 10, nullptr, cf, mi, mf, mi, mi, nullptr) == SV_ERR_LAUNCH);
    EXPECT(g_launches == before + 2);

    const size_t need = sv_verify_truncated_workspace_bytes(4, 3);
    EXPECT(need == 4 * (7 * sizeof(sv::LawRecord) + 64) && sizeof(sv::LawRecord) == 32);
    before = g_launches;
    EXPECT(sv_verify_truncated(F, 10, 8, F, 10, SV_F32, 10, ci, ci, 4, 3, &law, nullptr, 1, 2, mi, mi,
                               mf, mf, mf, mi, F, need - 1, nullptr) == SV_ERR_WORKSPACE);
    EXPECT(sv_verify_truncated(F, 10, 8, F, 10, SV_F32, 10, ci, ci, 2147483647, 64, &law, nullptr, 1,
                               2, mi, mi, mf, mf, mf, mi, F, need, nullptr) == SV_ERR_SHAPE);
    EXPECT(g_launches == before);
    EXPECT(sv_verify_truncated(F, 10, 8, F, 10, SV_F32, 10, ci, ci, 4, 3, &law, &law, 1, 2, mi, mi,
                               nullptr, nullptr, nullptr, nullptr, F, need, nullptr) ==
           SV_ERR_LAUNCH);
    EXPECT(g_launches == before + 1);

    for (const sv_dtype dt : {SV_BF16, SV_E4M3}) {
        for (const int dim : {64, 128, 256}) {
            const sv_cache c{F, F, dt, 100, 16, 2, dim, 32 * dim, 2 * dim, dim, nullptr, nullptr};
            before = g_launches;
            EXPECT(sv_cache_append(&c, ci, 4, F, F, 2 * dim, ci, ci, 8, ci, 2, mi, nullptr) ==
                   SV_ERR_LAUNCH);
            EXPECT(sv_cache_append(&c, ci, 4, F, F, 2 * dim - 8, ci, ci, 8, ci, 2, mi, nullptr) ==
                   SV_ERR_SHAPE);
            EXPECT(g_launches == before + 1);
            for (const int heads : {2, 6, 64, 512}) {
                for (const int k : {0, 7, 64}) {
                    for (const int n : {1, 3, 300}) {
                        for (const int pages : {0, 1, 100, 100000}) {
                            const size_t b = sv_cache_attend_workspace_bytes(n, k, heads, 2, dim,
                                                                             pages, 16);
                            before = g_launches;
                            const bool fits = (int64_t)n * heads * (k + 1) <= SV_MAX_ATTEND_SLOTS;
                            const sv_status st = sv_cache_attend(
                                &c, ci, pages, F, (int64_t)heads * dim, 1000, heads, ci, ci, n, k,
                                0.1f, F, (int64_t)heads * dim, nullptr, nullptr, b ? F : nullptr, b,
                                nullptr);
                            EXPECT(st == (fits ? SV_ERR_LAUNCH : SV_ERR_SHAPE));
                            EXPECT(g_launches == before + (fits ? 1 : 0));
                        }
                    }
                }
            }
        }
    }
    EXPECT(sv_cache_attend_workspace_bytes(2147483647, 64, 2147483647, 1, 64, 2147483647,
                                           2147483647) == 0);
    if (g_failures == 0) std::puts("serving checks passed");
    return g_failures != 0;
}
