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
    int parts;  // workgroups a row, a power of two
};
hipError_t launch_adjust(const AdjustArgs& a, hipStream_t stream);

constexpr int kAdjustTile = 512;         // ids
constexpr int kAdjustPartBytes = 32768;  // of a row, at most

// Workgroups a row: the power of two that makes some 8192 of them, with more than 2048
// ids each (a row of 4096 or fewer is one's), and no more ids than LDS holds.
inline int adjust_parts(int n_rows, int vocab, int esize) {
    const int tiles = (vocab + kAdjustTile - 1) / kAdjustTile;
    int p = 1;
    while ((int64_t)n_rows * p < 8192 && vocab > 2 * p * 2048) p *= 2;
    while ((tiles + p - 1) / p * kAdjustTile * esize > kAdjustPartBytes) p *= 2;
    return p;
}

}  // namespace sv
