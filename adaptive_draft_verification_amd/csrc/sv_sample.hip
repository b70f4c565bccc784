// sv_sample: one token a row under temperature, top-k, top-p and min-p.
// sv_law.h holds the mathematics; here one workgroup a row.
#include "sv_law.h"
#include "sv_launch.h"

namespace sv {
namespace {

template <sv_dtype DT, int NT>
__global__ __launch_bounds__(NT, NT == kWave ? 1 : 4) void sample_kernel(SampleArgs a) {
    __shared__ law::Smem<NT> sm;
    const int i = blockIdx.x;
    const law::Row<DT, NT> row(static_cast<const char*>(a.logits) +
                                   (int64_t)i * a.ld * law::Row<DT, NT>::kBytes, a.vocab);
    law::Settings set = law::settings(a.law, i, a.vocab);
    const float u = a.u[i];
    set.bad |= !(u >= 0.0f && u < 1.0f);
    const law::Result r = law::find_law<true>(row, set, sm);
    int tok = -1;
    if (!r.fault) tok = law::draw(row, r, u, sm);
    if (threadIdx.x == 0) {
        if (r.fault) raise_error(a.dev_error, r.fault);
        a.out_tokens[i] = tok;
        if (a.out_prob)
            a.out_prob[i] = r.fault ? -1.0f : (float)(r.w.raw(row.one(tok)) / r.total);
        if (a.out_support) a.out_support[i] = r.fault ? -1 : r.n;
    }
}

template <int NT>
void run(const SampleArgs& a, hipStream_t stream) {
    if (a.dtype == SV_BF16)
        sample_kernel<SV_BF16, NT><<<a.n_rows, NT, 0, stream>>>(a);
    else
        sample_kernel<SV_F32, NT><<<a.n_rows, NT, 0, stream>>>(a);
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, hipStream_t stream) {
    // Up to a workgroup for each CU, a row's own time counts: 1024 threads.
    // More rows share a CU: two workgroups of 512 threads, one summing while
    // the other waits for memory.  129,280 bf16 ids, 512 threads against 1024: 256
    // rows under top-p 74.7 us against 58.4, top-k 27.7 against 26.6, at a
    // temperature alone 44 against 39; 257 rows 76 against 77, 29 against 34, 66
    // against 70; 2048 rows 341 against 417, 125 against 167, 254 against 297;
    // 1024 rows of 256,000 fp32 ids under top-p 496 against 560.  (The exception
    // found: 257 .. 512 rows of settings mixed in turn, 74 against 57 us at 257.)
    // Rows of fewer than 8 ids: one wave each.
    if (a.vocab < 8) run<kWave>(a, stream);
    else if (a.n_rows > law::kCUs) run<512>(a, stream);
    else run<1024>(a, stream);
    return hipGetLastError();
}

}  // namespace sv
