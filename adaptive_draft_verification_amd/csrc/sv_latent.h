// Arguments, plan and launchers of the latent cache (internal; sv_latent_api.cpp
// validates before calling these).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "libspecverify.h"
#include "sv_serve.h"

namespace sv {

struct LatentAppendArgs {
    sv_latent_cache cache;
    const int32_t* page_table;
    int max_pages;
    const void* latent;
    int64_t latent_ld;
    const void* rope;
    int64_t rope_ld;
    const int32_t* row_req;
    const int32_t* row_pos;
    int n_rows;
    const int32_t* ctx_len;
    int n_req;
    int32_t* dev_error;
};
hipError_t launch_latent_append(const LatentAppendArgs& a, hipStream_t stream);

struct LatentAttendArgs {
    sv_latent_cache cache;
    const int32_t* page_table;
    int max_pages;
    const void* q;
    int64_t q_ld;
    int64_t q_rows;
    int n_heads;
    const int32_t* cu_rows;
    const int32_t* ctx_len;
    int n_req;
    int k_max;
    float scale;
    void* out;
    int64_t out_ld;
    float* out_lse;
    int32_t* dev_error;
    bool longest_first;  // requests by length (n_req <= 256)
    int page_shift;      // log2 of the page size, -1 if it is no power of two
    int slot_blocks, parts, part_min;  // LatentPlan's
    float* part_out;     // parts > 1: [n_req, k_max + 1, n_heads, parts, latent_dim]
    float* part_ml;      //            [..., parts, 2] m and sum
};
hipError_t launch_latent_attend(const LatentAttendArgs& a, hipStream_t stream);

// Positions of a part: whole tiles.
inline __host__ __device__ int latent_part_len(int len, int parts, int part_min) {
    const int even = ((len + parts - 1) / parts + 31) / 32 * 32;
    return even > part_min ? even : part_min;
}

// How a call is cut into workgroups: by host-known sizes alone.
struct LatentPlan {
    int slot_blocks;  // workgroups over a request's query slots, 64 each
    int parts;        // workgroups over the cached positions, at most
    int part_min;     // positions a part has at least
    LatentPlan(int n_req, int k_max, int n_heads, int64_t capacity) {
        const int64_t slots = (int64_t)(k_max + 1) * n_heads;
        constexpr int block = 64;
        slot_blocks = (int)((slots + block - 1) / block);
        // A part writes, and the join reads, four bytes a slot and latent dim, as much
        // as two positions' keys: four positions a slot keep that below the products'
        // time, and a workgroup has two tiles at least.
        const int64_t mine = slots < block ? slots : block;
        part_min = (int)((4 * mine + 63) / 64 * 64);
        // A CU holds one workgroup.  Few requests: as many as there are CUs, none twice.
        // Many: twice as many, so that short ones make room for long ones.  Measured the
        // one way and the other, n x 64 slots of 0 .. 4000 positions: n = 48 62 and 72 us, 64 70
        // and 90, 96 121 and 118, 128 135 and 139, 160 219 and 161, 192 222 and 187, 256 231 and
        // 200; n x 16 slots: 96 108 and 92, 192 219 and 165.  Where all have 4000 the first
        // is the better one up to 256 (64 93 and 116, 128 162 and 186, 192 250 and 307), but
        // lengths are not known here, and a server's differ.
        const int64_t groups = (int64_t)n_req * slot_blocks;
        const int64_t want = groups < 1 ? 1 : groups <= 64 ? 256 / groups
                                                           : (512 + groups - 1) / groups;
        const int64_t most = (capacity + part_min - 1) / part_min;
        const int64_t p = want < most ? want : most;
        parts = (int)(p < 1 ? 1 : p > 128 ? 128 : p);
    }
    int64_t grid(int n_req) const { return (int64_t)n_req * slot_blocks * parts; }
    size_t bytes(int n_req, int k_max, int n_heads, int latent_dim) const {
        if (parts == 1) return 0;
        return (size_t)n_req * n_heads * (k_max + 1) * parts * (latent_dim + 2) * sizeof(float);
    }
};

}  // namespace sv
