// Arguments, plan and launchers of attention over shared prefixes (internal;
// sv_shared_api.cpp validates before calling these).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "libspecverify.h"
#include "sv_serve.h"

namespace sv {

// Work on the prefixes is counted in tiles: 32 positions for a block of 128 query slots
// of one kv head.  Tiles lie in the order of kv heads, groups, the group's blocks and
// positions, and every workgroup takes an equal run of them, whatever blocks it falls
// into: one partial result for each, a segment.

// A group as the first launch finds it; one more behind the last has the totals.
struct SharedGroup {
    int64_t tile;   // tiles of a kv head before the group
    int32_t block;  // blocks before the group
    int32_t broken; // error bits: its requests are left alone
};

struct SharedTotals {
    int64_t run;     // tiles a workgroup takes
    int32_t chunks;  // workgroups with something to do
    int32_t pad;
};

struct SharedRequest {
    int32_t group;  // -1: of no group
    int32_t row;    // its first row among the group's
};

// The workgroups that share a block: the block's segment of workgroup c is number
// (block of all heads) + c.
struct SharedSpan {
    int32_t first, last;
};

struct SharedArgs {
    AttendArgs own;  // the positions behind the prefixes: the packed rows' own launch
    const int32_t* group_start;
    const int32_t* prefix_len;
    int n_groups;
    int chunks;              // SharedPlan's
    int32_t* first;          // [n_req] the first position of the request's own, -1: left alone
    SharedRequest* request;  // [n_req]
    SharedGroup* group;      // [n_groups + 1]
    SharedTotals* totals;
    SharedSpan* span;        // [kv heads, blocks]
    float* prefix_out;       // [segments, 128, head_dim]
    float* prefix_ml;        // [segments, 128, 2] m and sum
};
hipError_t launch_cache_attend_shared(const SharedArgs& a, hipStream_t stream);

// How the prefixes' launch is cut into workgroups: by host-known sizes alone.
struct SharedPlan {
    static constexpr int kSlots = 128, kTile = 32;
    // A run is four tiles at least (a segment's start, 7000 clocks or more, costs about as
    // much), and long enough that a block has 64 segments at most.  Equal runs instead of
    // parts of a length a block: 256 x 1 .. 8 rows behind 8192 positions 281 -> 218 us,
    // since 576 workgroups took turns on 512 places.
    static constexpr int kRunMin = 4, kSegments = 64;
    int64_t blocks;  // blocks of query slots over all groups and kv heads, at most
    int chunks;      // workgroups
    AttendPlan own;
    SharedPlan(int n_req, int n_groups, int k_max, int n_heads, int n_kv_heads, int head_dim,
               int esize, int64_t capacity)
        : own(n_req, k_max, n_heads, n_kv_heads, head_dim, esize, capacity) {
        if (own.parts > 64) own.parts = 64;  // the join takes 128 of both kinds
        // both kinds of workgroups are of one launch, with registers for two waves a SIMD
        if (own.slot_tiles * head_dim > 256) {
            own.slot_blocks *= own.slot_tiles * head_dim / 256;
            own.slot_tiles = 256 / head_dim;
        }
        const int64_t slots = (int64_t)n_req * (k_max + 1) * (n_heads / n_kv_heads);
        blocks = n_groups == 0 ? 0 : (slots / kSlots + n_groups) * n_kv_heads;
        // Two for each CU (one at dim 256, whose workgroups need all registers of a SIMD;
        // three would fit at dim 64 in 8 bits), fewer beside a lot of workgroups over own
        // positions; no more than there are runs.  256, 384, 512 and 768: 256 x 1 .. 8 rows
        // behind 8192 positions with up to 500 of their own 327, 314, 327, 326 us, of 8 bits
        // 329, 327, 318, 320; 256 x 1 row with one of their own 70, 77, 84, 87, with up to
        // 500 126, 134, 146, 153; 48 x 1 .. 8 of dim 64 in 8 bits 38.0, 39.2, 41.9, 44.4; 64 x
        // 1 .. 4 in eight groups, few workgroups over own positions, 29.8, 30.6, 31.8, 31.4.
        // So 384 is right where products take most of the call, and costs up to a tenth
        // where a request has one row.
        // (By the plan of two-byte caches: callers ask for the workspace without a type.)
        const bool many = AttendPlan(n_req, k_max, n_heads, n_kv_heads, head_dim, 2, capacity)
                              .grid(n_req, n_kv_heads) >= 512;
        chunks = head_dim == 256 ? 256 : many ? 384 : 512;
        const double runs = (double)blocks * ((capacity + kTile - 1) / kTile) / kRunMin + 8;
        if (runs < chunks) chunks = (int)runs & ~7;
    }
    int64_t segments() const { return blocks + chunks; }
    // The workspace: partial results of both launches, then what the first launch finds.
    size_t own_records(int n_req, int k_max, int n_heads) const {
        return (size_t)n_req * (k_max + 1) * n_heads * own.parts;
    }
    size_t bytes(int n_req, int n_groups, int k_max, int n_heads, int head_dim) const {
        return ((size_t)segments() * kSlots + own_records(n_req, k_max, n_heads)) *
                   (head_dim + 2) * sizeof(float) +
               (size_t)blocks * sizeof(SharedSpan) + sizeof(SharedTotals) +
               (size_t)(n_groups + 1) * sizeof(SharedGroup) +
               (size_t)n_req * (sizeof(SharedRequest) + sizeof(int32_t));
    }
};

}  // namespace sv
