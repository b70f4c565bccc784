// Arguments, plan and launchers of attention over shared prefixes (internal;
// sv_shared_api.cpp validates before calling these).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "libspecverify.h"
#include "sv_serve.h"

namespace sv {

// A block of a group's query slots, found by the first launch.
struct SharedBlock {
    int32_t group;  // -1: none
    int32_t index;
};

// What the first launch finds out about a request.
struct SharedRequest {
    int32_t group;   // -1: of no group
    int32_t record;  // where the records of its first row over the prefix are
};

struct SharedArgs {
    AttendArgs own;  // the positions behind the prefixes: the packed rows' own launch
    const int32_t* group_start;
    const int32_t* prefix_len;
    int n_groups;
    int prefix_blocks, prefix_parts, prefix_min;  // SharedPlan's
    int32_t* first;          // [n_req] the first position of the request's own, -1: left alone
    SharedRequest* request;  // [n_req]
    int32_t* broken;         // [n_groups] error bits
    SharedBlock* block;      // [prefix_blocks]
    float* prefix_out;       // [n_req, k_max + 1, n_heads, prefix_parts, head_dim]
    float* prefix_ml;        // [..., prefix_parts, 2] m and sum
};
hipError_t launch_cache_attend_shared(const SharedArgs& a, hipStream_t stream);

// How the prefixes' launch is cut into workgroups: by host-known sizes alone.
struct SharedPlan {
    static constexpr int kSlots = 128;  // of a workgroup
    int prefix_blocks;  // blocks of query slots over all groups, at most
    int prefix_parts;   // workgroups over a prefix's positions, at most
    int prefix_min;     // positions a part has at least
    AttendPlan own;
    SharedPlan(int n_req, int n_groups, int k_max, int n_heads, int n_kv_heads, int head_dim,
               int esize, int64_t capacity)
        : own(n_req, k_max, n_heads, n_kv_heads, head_dim, esize, capacity) {
        if (own.parts > 64) own.parts = 64;  // the join takes 128 of both kinds
        const int64_t slots = (int64_t)n_req * (k_max + 1) * (n_heads / n_kv_heads);
        prefix_blocks = (int)(slots / kSlots + n_groups);
        // Parts until there are some 1024 workgroups.  A part writes, and the join reads,
        // four bytes a slot and dim: 256 positions are eight tiles, a tenth of whose
        // products' time that takes.
        prefix_min = 256;
        const int64_t groups = (int64_t)prefix_blocks * n_kv_heads;
        const int64_t want = groups > 0 ? (1024 + groups - 1) / groups : 1;
        const int64_t most = (capacity + prefix_min - 1) / prefix_min;
        const int64_t p = want < most ? want : most;
        prefix_parts = (int)(p < 1 ? 1 : p > 64 ? 64 : p);
    }
    int64_t prefix_grid(int n_kv_heads) const {
        return (int64_t)prefix_blocks * n_kv_heads * prefix_parts;
    }
    // The workspace: records of both launches, then what the first launch finds.
    static size_t records(int n_req, int k_max, int n_heads) {
        return (size_t)n_req * (k_max + 1) * n_heads;
    }
    size_t float_count(int n_req, int k_max, int n_heads, int head_dim) const {
        return records(n_req, k_max, n_heads) * (size_t)(prefix_parts + own.parts) * (head_dim + 2);
    }
    size_t bytes(int n_req, int n_groups, int k_max, int n_heads, int head_dim) const {
        return float_count(n_req, k_max, n_heads, head_dim) * sizeof(float) +
               (size_t)n_req * (sizeof(int32_t) + sizeof(SharedRequest)) +
               (size_t)n_groups * sizeof(int32_t) + (size_t)prefix_blocks * sizeof(SharedBlock);
    }
};

}  // namespace sv
