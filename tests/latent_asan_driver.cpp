// Host-side checks of the history and logit calls, the latent cache and attention over
// shared prefixes under AddressSanitizer and UndefinedBehaviorSanitizer (test
// infrastructure, CPU only): their API files linked against stub launchers.  A call is
// refused without reaching a stub, or reaches it with arguments that a kernel could use:
// the stubs check the plans, and that the workspace holds all that they point into.
#include <cstdio>
#include <cstdint>
#include <limits>

#include "libspecverify.h"
#include "sv_latent.h"
#include "sv_launch.h"
#include "sv_logits.h"
#include "sv_shared.h"

static int g_launches = 0, g_failures = 0;
static const char* g_ws = nullptr;
static size_t g_ws_bytes = 0;

#define EXPECT(cond)                                                       \
    do {                                                                   \
        if (!(cond)) {                                                     \
            std::fprintf(stderr, "FAILED line %d: %s\n", __LINE__, #cond); \
            ++g_failures;                                                  \
        }                                                                  \
    } while (0)

// [p, p + bytes) lies in the workspace, on `align` bytes
static bool inside(const void* p, size_t bytes, size_t align) {
    const char* c = static_cast<const char*>(p);
    return c >= g_ws && c + bytes <= g_ws + g_ws_bytes &&
           reinterpret_cast<uintptr_t>(p) % align == 0;
}

namespace sv {
sv_status finish_launch(hipError_t e, hipStream_t) { return e == hipSuccess ? SV_OK : SV_ERR_LAUNCH; }
hipError_t launch_history_clear(const sv_history&, const int32_t*, int n, int32_t*, hipStream_t) {
    ++g_launches;
    EXPECT(n > 0 && (int64_t)n * 1024 < ((int64_t)1 << 32));
    return hipErrorNotSupported;
}
hipError_t launch_history_add(const HistoryAddArgs& a, hipStream_t) {
    ++g_launches;
    EXPECT(a.n > 0 && a.width > 0 && (int64_t)a.n * a.width < ((int64_t)1 << 32));
    return hipErrorNotSupported;
}
hipError_t launch_adjust(const AdjustArgs& a, hipStream_t) {
    ++g_launches;
    EXPECT(a.n_rows > 0 && a.parts > 0 && (int64_t)a.n_rows * a.parts * 256 < ((int64_t)1 << 32));
    EXPECT((a.parts & (a.parts - 1)) == 0);
    return hipErrorNotSupported;
}
hipError_t launch_latent_append(const LatentAppendArgs& a, hipStream_t) {
    ++g_launches;
    EXPECT((int64_t)a.n_rows * ((a.cache.latent_dim + SV_LATENT_ROPE) / 8) < ((int64_t)1 << 32));
    return hipErrorNotSupported;
}
hipError_t launch_latent_attend(const LatentAttendArgs& a, hipStream_t) {
    ++g_launches;
    const int64_t grid = (int64_t)a.n_req * a.slot_blocks * a.parts;
    EXPECT(grid > 0 && grid * 256 < ((int64_t)1 << 32));
    EXPECT(a.slot_blocks * 64 >= (a.k_max + 1) * a.n_heads);
    EXPECT(a.parts >= 1 && a.parts <= 128 && a.part_min % 32 == 0 && a.part_min > 0);
    const size_t records = (size_t)a.n_req * (a.k_max + 1) * a.n_heads * a.parts;
    if (a.parts > 1) {
        EXPECT(inside(a.part_out, records * a.cache.latent_dim * 4, 16));
        EXPECT(inside(a.part_ml, records * 8, 8));
    }
    const int64_t capacity = (int64_t)a.max_pages * a.cache.page_size;
    for (int64_t len : {(int64_t)1, capacity / 2, capacity})
        if (len > 0 && len < (1 << 30))
            EXPECT((int64_t)latent_part_len((int)len, a.parts, a.part_min) * a.parts >= len);
    return hipErrorNotSupported;
}
hipError_t launch_cache_attend_shared(const SharedArgs& s, hipStream_t) {
    ++g_launches;
    const AttendArgs& a = s.own;
    const int dim = a.cache.head_dim;
    const int64_t grid = (int64_t)a.n_req * a.cache.n_kv_heads * a.slot_blocks * a.parts;
    EXPECT(s.chunks >= 0 && s.chunks % 8 == 0 && s.chunks <= 512);
    EXPECT(s.n_groups == 0 || s.chunks > 0);
    EXPECT(grid > 0 && (grid + s.chunks) * 256 < ((int64_t)1 << 32));
    EXPECT(a.slot_blocks * 16 * a.slot_tiles >= (a.k_max + 1) * a.group);
    EXPECT(a.slot_tiles * dim <= 256 && a.parts >= 1 && a.parts <= 64);
    const size_t slots = (size_t)a.n_req * (a.k_max + 1) * a.group;
    const size_t blocks = s.n_groups == 0 ? 0 : (slots / 128 + s.n_groups) * a.cache.n_kv_heads;
    const size_t segments = (blocks + s.chunks) * 128;
    const size_t own = (size_t)a.n_req * (a.k_max + 1) * a.n_heads * a.parts;
    EXPECT(inside(s.prefix_out, segments * dim * 4, 16));
    EXPECT(inside(s.prefix_ml, segments * 8, 8));
    EXPECT(inside(a.part_out, own * dim * 4, 16));
    EXPECT(inside(a.part_ml, own * 8, 8));
    EXPECT(inside(s.group, (s.n_groups + 1) * sizeof(SharedGroup), 8));
    EXPECT(inside(s.totals, sizeof(SharedTotals), 8));
    EXPECT(inside(s.span, blocks * sizeof(SharedSpan), 4));
    EXPECT(inside(s.request, a.n_req * sizeof(SharedRequest), 4));
    EXPECT(inside(s.first, a.n_req * sizeof(int32_t), 4) && a.first == s.first);
    // one behind the other
    const char* at[] = {reinterpret_cast<const char*>(s.prefix_out),
                        reinterpret_cast<const char*>(a.part_out),
                        reinterpret_cast<const char*>(s.prefix_ml),
                        reinterpret_cast<const char*>(a.part_ml),
                        reinterpret_cast<const char*>(s.group),
                        reinterpret_cast<const char*>(s.totals),
                        reinterpret_cast<const char*>(s.span),
                        reinterpret_cast<const char*>(s.request),
                        reinterpret_cast<const char*>(s.first)};
    const size_t size[] = {segments * dim * 4, own * dim * 4, segments * 8, own * 8,
                           (s.n_groups + 1) * sizeof(SharedGroup), sizeof(SharedTotals),
                           blocks * sizeof(SharedSpan), a.n_req * sizeof(SharedRequest)};
    for (int i = 0; i < 8; ++i) EXPECT(at[i] + size[i] <= at[i + 1]);
    return hipErrorNotSupported;
}
}  // namespace sv

int main() {
    alignas(16) static float fake[64];
    void* F = fake;
    int32_t* mi = reinterpret_cast<int32_t*>(fake);
    const int32_t* ci = mi;
    const float* cf = fake;

    const sv_history h{mi, mi, mi, 4, 100, 8};
    int before = g_launches;
    EXPECT(sv_history_add(&h, ci, ci, 3, 2, 4, 0, mi, nullptr) == SV_ERR_SHAPE);
    EXPECT(sv_history_add(&h, ci, ci, std::numeric_limits<int64_t>::max(), 1 << 20, 1, 0, mi,
                          nullptr) == SV_ERR_SHAPE);
    EXPECT(sv_history_clear(&h, ci, std::numeric_limits<int32_t>::max(), mi, nullptr) ==
           SV_ERR_SHAPE);
    EXPECT(g_launches == before);
    EXPECT(sv_history_add(&h, ci, ci, 4, 2, 4, 0, mi, nullptr) == SV_ERR_LAUNCH);
    EXPECT(sv_history_clear(&h, nullptr, 4, nullptr, nullptr) == SV_ERR_LAUNCH);
    EXPECT(g_launches == before + 2);
    const sv_penalties pen{cf, cf, cf};
    for (const sv_dtype dt : {SV_F32, SV_BF16})
        for (const int vocab : {1, 100, 128255, SV_MAX_VOCAB})
            for (const int rows : {1, 2, 2048, 1 << 20}) {
                const sv_history hv{mi, mi, mi, 4, vocab, 8};
                before = g_launches;
                const sv_status st =
                    sv_adjust_logits(F, vocab, F, vocab, rows, dt, vocab, ci, ci, 4, 3, ci, &hv,
                                     nullptr, &pen, nullptr, nullptr, mi, nullptr);
                EXPECT(st == SV_ERR_LAUNCH || st == SV_ERR_SHAPE);
                EXPECT(g_launches == before + (st == SV_ERR_LAUNCH));
                EXPECT(st == SV_ERR_LAUNCH || rows > 2048);
                EXPECT(sv_adjust_logits(F, std::numeric_limits<int64_t>::max(), F, vocab, rows, dt,
                                        vocab, ci, ci, 4, 3, ci, nullptr, nullptr, nullptr, nullptr,
                                        nullptr, mi, nullptr) == SV_ERR_SHAPE);
            }

    for (const sv_dtype dt : {SV_BF16, SV_E4M3}) {
        for (const int rank : {256, 512}) {
            const sv_latent_cache c{F, dt, 100, 16, rank, 16 * (rank + 64), rank + 64, nullptr};
            before = g_launches;
            EXPECT(sv_latent_append(&c, ci, 4, F, rank, F, 64, ci, ci, 8, ci, 2, mi, nullptr) ==
                   SV_ERR_LAUNCH);
            EXPECT(sv_latent_append(&c, ci, 4, F, rank - 8, F, 64, ci, ci, 8, ci, 2, mi, nullptr) ==
                   SV_ERR_SHAPE);
            EXPECT(sv_latent_append(&c, ci, 4, F, rank, F, 56, ci, ci, 8, ci, 2, mi, nullptr) ==
                   SV_ERR_SHAPE);
            EXPECT(g_launches == before + 1);
            for (const int heads : {1, 5, 128, 1000})
                for (const int k : {0, 7, 64})
                    for (const int n : {1, 3, 300})
                        for (const int pages : {0, 1, 100, 100000}) {
                            const size_t b =
                                sv_latent_attend_workspace_bytes(n, k, heads, rank, pages, 16);
                            g_ws = b ? reinterpret_cast<const char*>((uintptr_t)1 << 40) : nullptr;
                            g_ws_bytes = b;
                            before = g_launches;
                            const bool fits = (int64_t)n * heads * (k + 1) <= SV_MAX_ATTEND_SLOTS;
                            const sv_status st = sv_latent_attend(
                                &c, ci, pages, F, (int64_t)heads * (rank + 64), 1000, heads, ci, ci,
                                n, k, 0.1f, F, (int64_t)heads * rank, nullptr, nullptr,
                                const_cast<char*>(g_ws), b, nullptr);
                            EXPECT(st == (fits ? SV_ERR_LAUNCH : SV_ERR_SHAPE));
                            EXPECT(g_launches == before + (fits ? 1 : 0));
                        }
        }
        for (const int dim : {64, 128, 256}) {
            const sv_cache c{F, F, dt, 100, 16, 2, dim, 32 * dim, 2 * dim, dim, nullptr, nullptr};
            for (const int heads : {2, 6, 64, 512})
                for (const int k : {0, 7, 64})
                    for (const int n : {1, 3, 300})
                        for (const int groups : {0, 1, 3, 300})
                            for (const int pages : {0, 1, 100, 100000, 100000000}) {
                                const size_t b = sv_cache_attend_shared_workspace_bytes(
                                    n, groups, k, heads, 2, dim, pages, 16);
                                g_ws = reinterpret_cast<const char*>((uintptr_t)1 << 40);
                                g_ws_bytes = b;
                                before = g_launches;
                                const bool fits = groups <= n &&
                                                  (int64_t)n * heads * (k + 1) <=
                                                      SV_MAX_ATTEND_SLOTS;
                                auto call = [&](size_t bytes) {
                                    return sv_cache_attend_shared(
                                        &c, ci, pages, F, (int64_t)heads * dim, 1000, heads, ci, ci,
                                        n, k, groups ? ci : nullptr, groups ? ci : nullptr, groups,
                                        0.1f, F, (int64_t)heads * dim, nullptr, nullptr,
                                        const_cast<char*>(g_ws), bytes, nullptr);
                                };
                                EXPECT((b > 0) == fits);
                                EXPECT(call(b) == (fits ? SV_ERR_LAUNCH : SV_ERR_SHAPE));
                                EXPECT(g_launches == before + (fits ? 1 : 0));
                                // an 8-bit cache may need less
                                if (fits && dt == SV_BF16)
                                    EXPECT(call(b - 1) == SV_ERR_WORKSPACE);
                            }
        }
    }
    // the size asked for does not know the cache's type: it has to do for either
    for (const sv_dtype dt : {SV_BF16, SV_E4M3})
        for (const int heads : {1, 8, 16})
            for (const int k : {0, 3, 7})
                for (int n = 1; n < 200; n += n < 20 ? 1 : 17)
                    for (const int pages : {16, 128, 512, 4096}) {
                        const sv_cache c{F, F, dt, 100, 16, 1, 64, 1024, 64, 64, nullptr, nullptr};
                        const size_t b =
                            sv_cache_attend_shared_workspace_bytes(n, n, k, heads, 1, 64, pages, 16);
                        g_ws = reinterpret_cast<const char*>((uintptr_t)1 << 40);
                        g_ws_bytes = b;
                        EXPECT(sv_cache_attend_shared(&c, ci, pages, F, heads * 64, 1000, heads, ci,
                                                      ci, n, k, ci, ci, n, 0.1f, F, heads * 64,
                                                      nullptr, nullptr, const_cast<char*>(g_ws), b,
                                                      nullptr) == SV_ERR_LAUNCH);
                    }
    EXPECT(sv_latent_attend_workspace_bytes(2147483647, 64, 2147483647, 512, 2147483647,
                                            2147483647) == 0);
    EXPECT(sv_cache_attend_shared_workspace_bytes(2147483647, 2147483647, 64, 2147483647, 1, 64,
                                                  2147483647, 2147483647) == 0);
    if (g_failures == 0) std::puts("latent and shared checks passed");
    return g_failures != 0;
}
