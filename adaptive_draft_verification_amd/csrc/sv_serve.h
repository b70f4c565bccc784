// Arguments and launchers of the paged cache and of the truncated laws
// (internal; sv_cache_api.cpp and sv_sample_api.cpp validate before calling
// these).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "libspecverify.h"

namespace sv {

struct AppendArgs {
    sv_cache cache;
    const int32_t* page_table;
    int max_pages;
    const void* k;
    const void* v;
    int64_t kv_ld;
    const int32_t* row_req;
    const int32_t* row_pos;
    int n_rows;
    const int32_t* ctx_len;
    int n_req;
    int32_t* dev_error;
};
hipError_t launch_cache_append(const AppendArgs& a, hipStream_t stream);

struct AttendArgs {
    sv_cache cache;
    const int32_t* page_table;
    int max_pages;
    const void* q;
    int64_t q_ld;
    int64_t q_rows;
    int n_heads;
    int group;  // query heads per kv head
    const int32_t* cu_rows;
    const int32_t* ctx_len;
    int n_req;
    int k_max;
    float scale;
    void* out;
    int64_t out_ld;
    float* out_lse;
    int32_t* dev_error;
    int xcd_run;                         // neighbouring heads that share cache lines
    bool longest_first;                  // requests by length (n_req <= 256)
    int page_shift;                      // log2 of the page size, -1 if it is no power of two
    int slot_tiles, slot_blocks, parts, part_min;  // AttendPlan's
    float* part_out;                     // parts > 1: [n_req, n_heads, k_max + 1, parts, head_dim]
    float* part_ml;                      //            [..., parts, 2] m and sum
    const int32_t* first;                // [n_req] the first position of the request's own, where a
                                         // prefix is shared
};
hipError_t launch_cache_attend(const AttendArgs& a, hipStream_t stream);

// Positions in each part of a request's length: a multiple of 128 (four waves
// of 32), no fewer than part_min.
inline __host__ __device__ int part_len(int len, int parts, int part_min) {
    const int even = ((len + parts - 1) / parts + 127) / 128 * 128;
    return even > part_min ? even : part_min;
}

// How an attend call is cut into workgroups: by host-known sizes alone.
struct AttendPlan {
    int slot_tiles;   // 16-slot tiles a workgroup takes: 1, 2 or 4
    int slot_blocks;  // workgroups over a (request, kv head)'s query slots
    int parts;        // workgroups over the cached positions, at most
    int part_min;     // positions a part has at least
    AttendPlan(int n_req, int k_max, int n_heads, int n_kv_heads, int head_dim, int esize,
               int64_t capacity) {
        const int slots = (k_max + 1) * (n_heads / n_kv_heads);
        slot_tiles = slots <= 16 || head_dim > 128 ? 1 : slots <= 32 ? 2 : 4;
        slot_blocks = (slots + 16 * slot_tiles - 1) / (16 * slot_tiles);
        // a part writes, and the join reads, 4 bytes a slot and dim, against 2
        // esize bytes a position and dim: 32 positions a slot (64 for one-byte
        // caches) keep that to a sixteenth of the reads
        const int block = slots < 16 * slot_tiles ? slots : 16 * slot_tiles;
        part_min = (32 * (esize == 1 ? 2 : 1) * block + 127) / 128 * 128;
        // Parts until there are about 1024 workgroups, four for a CU, at most 128
        // (two factors a lane of the join).  Measured with 256, 512, 1024 and 2048:
        // e4m3, whose conversions want waves, 3 requests of 100,005 positions 198,
        // 182, 154, 165 us, 16 of 4001 42, 30, 36, 39; bf16, 1 request of 16,001
        // 20, 22, 29, 29, 16 of 4001 47, 50, 49, 55, 64 of 2001 102, 102, 107, 112,
        // 1 of 131,001 108, 110, 117, 116.  The cap leaves CUs idle at one kv head
        // (131,001 positions: 31 us, 2.2 TB/s; two heads 37, 3.6; eight 117, 4.6).
        // Lengths are not known here: a batch that fills the chip is not split,
        // and waits for a request much longer than the rest (255 of up to 2000
        // positions 200 us, with one of 32,000 585, of 100,000 1550).
        const int64_t groups = (int64_t)n_req * n_kv_heads * slot_blocks;
        const int64_t want = groups > 0 ? (1024 + groups - 1) / groups : 1;
        const int64_t most = (capacity + part_min - 1) / part_min;
        const int64_t p = want < most ? want : most;
        parts = (int)(p < 1 ? 1 : p > 128 ? 128 : p);
    }
    int64_t grid(int n_req, int n_kv_heads) const {
        return (int64_t)n_req * n_kv_heads * slot_blocks * parts;
    }
    size_t bytes(int n_req, int k_max, int n_heads, int head_dim) const {
        if (parts == 1) return 0;
        return (size_t)n_req * n_heads * (k_max + 1) * parts * (head_dim + 2) * sizeof(float);
    }
};

struct SampleArgs {
    const void* logits;
    int64_t ld;
    int n_rows;
    sv_dtype dtype;
    int vocab;
    sv_sampling law;
    const float* u;
    int32_t* out_tokens;
    float* out_prob;
    int32_t* out_support;
    int32_t* dev_error;
};
hipError_t launch_sample(const SampleArgs& a, hipStream_t stream);

// One row's law, from the first launch of sv_verify_truncated to the second.
struct LawRecord {
    double total;    // the support's weight
    float top;       // the largest logit
    float zc;        // the support's last logit and last id of it
    int32_t cid;
    int32_t fault;   // SV_DEV_* bits
    double drafted;  // the weight of the position's draft id (0: outside)
};

struct VerifyTruncatedArgs {
    const void* target;
    int64_t target_ld;
    int64_t target_rows;
    const void* draft;
    int64_t draft_ld;
    sv_dtype dtype;
    int vocab;
    const int32_t* draft_tokens;
    const int32_t* cu_rows;
    int n_req;
    int k_max;
    sv_sampling target_law;
    sv_sampling draft_law;
    uint64_t seed;
    uint64_t step;
    int32_t* out_tokens;
    int32_t* out_accepted;
    float* out_p_draft;
    float* out_q_draft;
    float* out_residual_mass;
    int32_t* dev_error;
    LawRecord* laws;  // [n_req, 2 k_max + 1]: target rows 0 .. k_max, draft rows
    double* sums;     // [n_req, kVerifyParts]: of the row the token at L is drawn from
};
constexpr int kVerifyParts = 8;
hipError_t launch_verify_truncated(const VerifyTruncatedArgs& a, hipStream_t stream);

}  // namespace sv
