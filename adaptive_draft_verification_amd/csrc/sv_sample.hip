// sv_sample: one token a row under temperature, top-k, top-p and min-p.
// sv_law.h holds the mathematics; here one 1024-thread workgroup a row.
#include "sv_law.h"
#include "sv_launch.h"

namespace sv {
namespace {

template <sv_dtype DT>
__global__ __launch_bounds__(law::kThreads) void sample_kernel(SampleArgs a) {
    __shared__ law::Smem sm;
    const int i = blockIdx.x;
    const law::Row<DT> row(static_cast<const char*>(a.logits) +
                               (int64_t)i * a.ld * law::Row<DT>::kBytes, a.vocab);
    law::Settings set = law::settings(a.law, i, a.vocab);
    const float u = a.u[i];
    set.bad |= !(u >= 0.0f && u < 1.0f);
    const law::Result r = law::find_law<DT>(row, set, sm);
    int tok = -1;
    if (!r.fault) tok = law::draw<DT>(row, r, u, sm);
    if (threadIdx.x == 0) {
        if (r.fault) raise_error(a.dev_error, r.fault);
        a.out_tokens[i] = tok;
        if (a.out_prob)
            a.out_prob[i] = r.fault ? -1.0f : (float)(r.w.raw(row.one(tok)) / r.total);
        if (a.out_support) a.out_support[i] = r.fault ? -1 : r.n;
    }
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, hipStream_t stream) {
    if (a.dtype == SV_BF16)
        sample_kernel<SV_BF16><<<a.n_rows, law::kThreads, 0, stream>>>(a);
    else
        sample_kernel<SV_F32><<<a.n_rows, law::kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace sv
