// C ABI of sampling and verification under truncated laws: host-side
// validation, then launches on the caller's stream.  Every check runs before
// any HIP call.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "libspecverify.h"
#include "sv_launch.h"
#include "sv_serve.h"

namespace {

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

sv_sampling law_of(const sv_sampling* l) { return l != nullptr ? *l : sv_sampling{}; }

bool value_aligned(const void* p, sv_dtype dtype) {
    return (reinterpret_cast<uintptr_t>(p) & (dtype == SV_BF16 ? 1 : 3)) == 0;
}

}  // namespace

extern "C" {

sv_status sv_sample(const void* logits, int64_t ld, int32_t n_rows, sv_dtype dtype,
                    int32_t vocab, const sv_sampling* law, const float* u, int32_t* out_tokens,
                    float* out_prob, int32_t* out_support, int32_t* dev_error, void* stream) {
    if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
    if (n_rows < 0 || n_rows > SV_MAX_SAMPLE_ROWS) return SV_ERR_SHAPE;
    if (vocab < 1 || vocab > SV_MAX_VOCAB || ld < vocab) return SV_ERR_SHAPE;
    if (n_rows == 0) return SV_OK;
    if (logits == nullptr || u == nullptr || out_tokens == nullptr) return SV_ERR_NULL;
    if (!value_aligned(logits, dtype)) return SV_ERR_SHAPE;
    if ((double)n_rows * (double)ld > 2.0e18) return SV_ERR_SHAPE;
    const sv::SampleArgs a{logits, ld,         n_rows,   dtype,       vocab,    law_of(law),
                           u,      out_tokens, out_prob, out_support, dev_error};
    const hipError_t e = sv::launch_sample(a, as_stream(stream));
    return sv::finish_launch(e, as_stream(stream));
}

size_t sv_verify_truncated_workspace_bytes(int32_t n_req, int32_t k_max) {
    if (n_req < 0 || k_max < 0 || k_max > SV_MAX_DRAFT ||
        (int64_t)n_req * (2 * k_max + 1) > SV_MAX_VERIFY_SLOTS)
        return 0;
    return (size_t)n_req * ((2 * k_max + 1) * sizeof(sv::LawRecord) +
                            sv::kVerifyParts * sizeof(double));
}

sv_status sv_verify_truncated(const void* target_logits, int64_t target_ld, int64_t target_rows,
                              const void* draft_logits, int64_t draft_ld, sv_dtype dtype,
                              int32_t vocab, const int32_t* draft_tokens, const int32_t* cu_rows,
                              int32_t n_req, int32_t k_max, const sv_sampling* target_law,
                              const sv_sampling* draft_law, uint64_t seed, uint64_t step,
                              int32_t* out_tokens, int32_t* out_accepted, float* out_p_draft,
                              float* out_q_draft, float* out_residual_mass, int32_t* dev_error,
                              void* ws, size_t ws_bytes, void* stream) {
    if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
    if (n_req < 0 || k_max < 0 || k_max > SV_MAX_DRAFT) return SV_ERR_SHAPE;
    if ((int64_t)n_req * (2 * k_max + 1) > SV_MAX_VERIFY_SLOTS) return SV_ERR_SHAPE;
    if (vocab < 1 || vocab > SV_MAX_VOCAB || target_rows < 0 || target_ld < vocab)
        return SV_ERR_SHAPE;
    if (k_max > 0 && draft_ld < vocab) return SV_ERR_SHAPE;
    if (n_req == 0) return SV_OK;
    if (target_logits == nullptr || cu_rows == nullptr || out_tokens == nullptr ||
        out_accepted == nullptr)
        return SV_ERR_NULL;
    if (k_max > 0 && (draft_tokens == nullptr || draft_logits == nullptr)) return SV_ERR_NULL;
    if (!value_aligned(target_logits, dtype) || !value_aligned(draft_logits, dtype))
        return SV_ERR_SHAPE;
    // the largest element offset a kernel may form must fit int64
    if ((double)target_rows * (double)target_ld > 2.0e18 ||
        (double)n_req * k_max * (double)draft_ld > 2.0e18)
        return SV_ERR_SHAPE;
    const size_t need = sv_verify_truncated_workspace_bytes(n_req, k_max);
    if (ws == nullptr || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 7) != 0)
        return SV_ERR_WORKSPACE;
    const sv::VerifyTruncatedArgs a{target_logits, target_ld, target_rows, draft_logits, draft_ld,
                                    dtype, vocab, draft_tokens, cu_rows, n_req, k_max,
                                    law_of(target_law), law_of(draft_law), seed, step,
                                    out_tokens, out_accepted, out_p_draft, out_q_draft,
                                    out_residual_mass, dev_error,
                                    static_cast<sv::LawRecord*>(ws),
                                    reinterpret_cast<double*>(
                                        static_cast<sv::LawRecord*>(ws) +
                                        (size_t)n_req * (2 * k_max + 1))};
    const hipError_t e = sv::launch_verify_truncated(a, as_stream(stream));
    return sv::finish_launch(e, as_stream(stream));
}

}  // extern "C"
