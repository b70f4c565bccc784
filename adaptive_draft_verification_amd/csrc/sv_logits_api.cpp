// C ABI of the history and of the adjusted logits: host-side validation, then
// launches on the caller's stream.  Every check runs before any HIP call.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "libspecverify.h"
#include "sv_launch.h"
#include "sv_logits.h"

namespace {

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

sv_status check_history(const sv_history& h) {
    if (h.n_slots < 0 || h.cap < 0 || h.vocab < 1 || h.vocab > SV_MAX_VOCAB) return SV_ERR_SHAPE;
    return SV_OK;
}

bool history_null(const sv_history& h) {
    return h.counts == nullptr || h.n_seen == nullptr || (h.cap > 0 && h.seen == nullptr);
}

// Rows that are the same, or that share no byte.
bool overlap_ok(const void* a, int64_t a_ld, const void* b, int64_t b_ld, int64_t rows, int64_t width,
                int64_t esize) {
    if (a == b && a_ld == b_ld) return true;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    const uintptr_t a1 = a0 + (uintptr_t)(((rows - 1) * a_ld + width) * esize);
    const uintptr_t b1 = b0 + (uintptr_t)(((rows - 1) * b_ld + width) * esize);
    return a1 <= b0 || b1 <= a0;
}

}  // namespace

extern "C" {

sv_status sv_history_clear(const sv_history* history, const int32_t* slots, int32_t n,
                           int32_t* dev_error, void* stream) {
    if (history == nullptr) return SV_ERR_NULL;
    const sv_status hs = check_history(*history);
    if (hs != SV_OK) return hs;
    if (n < 0 || (int64_t)n * 1024 > SV_MAX_HISTORY_TOKENS) return SV_ERR_SHAPE;
    if (n == 0) return SV_OK;
    if (history_null(*history)) return SV_ERR_NULL;
    const hipError_t e = sv::launch_history_clear(*history, slots, n, dev_error, as_stream(stream));
    return sv::finish_launch(e, as_stream(stream));
}

sv_status sv_history_add(const sv_history* history, const int32_t* slots, const int32_t* tokens,
                         int64_t tokens_ld, int32_t n, int32_t width, int32_t in_prompt,
                         int32_t* dev_error, void* stream) {
    if (history == nullptr) return SV_ERR_NULL;
    const sv_status hs = check_history(*history);
    if (hs != SV_OK) return hs;
    if (n < 0 || width < 0 || tokens_ld < width) return SV_ERR_SHAPE;
    // a row's last workgroup may be one id's
    if ((int64_t)n * (((int64_t)width + 255) / 256 * 256) > SV_MAX_HISTORY_TOKENS)
        return SV_ERR_SHAPE;
    if (n == 0 || width == 0) return SV_OK;
    if (history_null(*history) || tokens == nullptr) return SV_ERR_NULL;
    if ((double)n * (double)tokens_ld > 2.0e18) return SV_ERR_SHAPE;
    const sv::HistoryAddArgs a{*history, slots, tokens, tokens_ld, n, width, in_prompt != 0,
                               dev_error};
    const hipError_t e = sv::launch_history_add(a, as_stream(stream));
    return sv::finish_launch(e, as_stream(stream));
}

sv_status sv_adjust_logits(const void* logits, int64_t ld, void* out, int64_t out_ld,
                           int32_t n_rows, sv_dtype dtype, int32_t vocab, const int32_t* row_req,
                           const int32_t* row_pos, int32_t n_req, int32_t k_max,
                           const int32_t* draft_tokens, const sv_history* history,
                           const int32_t* slots, const sv_penalties* penalties,
                           const sv_bias* bias, const sv_token_mask* mask, int32_t* dev_error,
                           void* stream) {
    if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
    if (n_rows < 0 || n_rows > SV_MAX_SAMPLE_ROWS) return SV_ERR_SHAPE;
    if (vocab < 1 || vocab > SV_MAX_VOCAB || ld < vocab || out_ld < vocab) return SV_ERR_SHAPE;
    if (n_req < 0 || k_max < 0 || k_max > SV_MAX_DRAFT) return SV_ERR_SHAPE;
    if (history != nullptr) {
        const sv_status hs = check_history(*history);
        if (hs != SV_OK) return hs;
        if (history->vocab != vocab) return SV_ERR_SHAPE;
    }
    if (bias != nullptr && bias->n_entries < 0) return SV_ERR_SHAPE;
    if (mask != nullptr &&
        (mask->n_masks < 0 || mask->ld < ((int64_t)vocab + 31) / 32 ||
         (double)mask->n_masks * (double)mask->ld > 2.0e18))
        return SV_ERR_SHAPE;
    if (n_rows == 0) return SV_OK;
    if (logits == nullptr || out == nullptr) return SV_ERR_NULL;
    if ((row_req == nullptr) != (row_pos == nullptr)) return SV_ERR_NULL;
    if (row_req == nullptr && n_rows > n_req) return SV_ERR_SHAPE;
    if (k_max > 0 && penalties != nullptr && draft_tokens == nullptr) return SV_ERR_NULL;
    if (history != nullptr && penalties != nullptr && history_null(*history)) return SV_ERR_NULL;
    if (bias != nullptr && (bias->start == nullptr ||
                            (bias->n_entries > 0 && (bias->ids == nullptr || bias->values == nullptr))))
        return SV_ERR_NULL;
    if (mask != nullptr && mask->n_masks > 0 && mask->bits == nullptr) return SV_ERR_NULL;
    const uintptr_t esize = dtype == SV_BF16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(logits) % esize != 0 ||
        reinterpret_cast<uintptr_t>(out) % esize != 0)
        return SV_ERR_SHAPE;
    // the largest byte offset a kernel may form must fit int64
    if ((double)n_rows * (double)ld > 2.0e18 || (double)n_rows * (double)out_ld > 2.0e18)
        return SV_ERR_SHAPE;
    if (!overlap_ok(logits, ld, out, out_ld, n_rows, vocab, (int64_t)esize)) return SV_ERR_SHAPE;
    const int parts = sv::adjust_parts(n_rows, vocab, (int)esize);
    if ((int64_t)n_rows * parts > SV_MAX_ADJUST_PARTS) return SV_ERR_SHAPE;
    const sv::AdjustArgs a{logits, ld, out, out_ld, n_rows, dtype, vocab, row_req, row_pos, n_req,
                           k_max, draft_tokens,
                           history != nullptr && penalties != nullptr ? *history : sv_history{},
                           slots, penalties != nullptr,
                           penalties != nullptr ? *penalties : sv_penalties{},
                           bias != nullptr ? *bias : sv_bias{}, mask != nullptr,
                           mask != nullptr ? *mask : sv_token_mask{}, dev_error,
                           parts};
    const hipError_t e = sv::launch_adjust(a, as_stream(stream));
    return sv::finish_launch(e, as_stream(stream));
}

}  // extern "C"
