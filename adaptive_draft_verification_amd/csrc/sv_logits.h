// Arguments and launchers of the history and of the adjusted logits (internal;
// sv_logits_api.cpp validates before calling these).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "libspecverify.h"

namespace sv {

hipError_t launch_history_clear(const sv_history& h, const int32_t* slots, int n,
                                int32_t* dev_error, hipStream_t stream);

struct HistoryAddArgs {
    sv_history history;
    const int32_t* slots;
    const int32_t* tokens;
    int64_t tokens_ld;
    int n;
    int width;
    bool in_prompt;
    int32_t* dev_error;
};
hipError_t launch_history_add(const HistoryAddArgs& a, hipStream_t stream);

struct AdjustArgs {
    const void* logits;
    int64_t ld;
    void* out;
    int64_t out_ld;
    int n_rows;
    sv_dtype dtype;
    int vocab;
    const int32_t* row_req;
    const int32_t* row_pos;
    int n_req;
    int k_max;
    const int32_t* draft_tokens;
    sv_history history;  // counts = NULL: none
    const int32_t* slots;
    bool penalised;
    sv_penalties penalties;
    sv_bias bias;        // n_entries = 0: none
    bool masked;
    sv_token_mask mask;
    int32_t* dev_error;
    int parts;     // workgroups a row
    int part_len;  // ids of each, a multiple of 32
};
hipError_t launch_adjust(const AdjustArgs& a, hipStream_t stream);

// Ids a workgroup takes: rows are cut until there are some 2048 workgroups, not
// below 4096 ids.
inline int adjust_part_len(int n_rows, int vocab) {
    const int64_t want = n_rows > 0 ? (2048 + n_rows - 1) / n_rows : 1;
    const int64_t even = ((vocab + want - 1) / want + 31) / 32 * 32;
    return (int)(even < 4096 ? 4096 : even);
}

}  // namespace sv
