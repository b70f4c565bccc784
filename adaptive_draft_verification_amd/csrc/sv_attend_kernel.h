// The attention kernel of the paged cache (gfx950, wave64): sv_cache_attend's, and
// sv_cache_attend_shared's for the positions behind a request's prefix.
#pragma once

#include "sv_attend.h"
#include "sv_device.h"
#include "sv_serve.h"

namespace sv {
namespace {

// A request's query slots of one kv head are its rows times the G query heads
// that share it (slot i: row i / G, head h G + i % G).  One workgroup of four
// waves takes up to 16 MT slots of a (request, kv head) over one part of the
// cached positions; its waves take the part's 32-position tiles in turn, each
// with its own running maximum and sum, and are merged through LDS.  Parts
// are merged by a second launch.  Keys and values are read once per 16 MT
// slots, straight into registers in the operand layouts of
// v_mfma_f32_16x16x32_bf16, without LDS:
//   S^T = K Q^T: operand A holds 16 positions (lane % 16) by 32 dims, B 16
//   slots by the same dims, so a lane ends with the scores of ONE slot
//   (lane % 16) at positions 4 g .. 4 g + 3 of each 16 (g = lane / 16);
//   O^T = V^T P^T: B's lane holds 8 positions of one slot: exactly the scores
//   the lane has from two 16-position products, in the order they are in.  A
//   needs 8 positions of one dim a lane: the lane loads dims c D/16 .. of its
//   group's 8 positions (16 lanes read one position's whole row) and swaps
//   halves of register pairs.  Product i of D/16 makes dims (row D/16 + i), so
//   a lane's accumulators are D/4 consecutive dims of its slot.
// The order of the contracted index is free as long as both operands agree.

template <int N>
struct Words {
    uint32_t w[N];
};

template <int N>
__device__ __forceinline__ Words<N> load_words(const void* p) {
    Words<N> out;
    if constexpr (N == 1) {
        out.w[0] = *static_cast<const uint32_t*>(p);
    } else if constexpr (N == 2) {
        const uint2 v = *static_cast<const uint2*>(p);
        out.w[0] = v.x;
        out.w[1] = v.y;
    } else {
        static_assert(N % 4 == 0, "1, 2 or a multiple of 4 words");
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 v = static_cast<const uint4*>(p)[i];
            out.w[4 * i] = v.x;
            out.w[4 * i + 1] = v.y;
            out.w[4 * i + 2] = v.z;
            out.w[4 * i + 3] = v.w;
        }
    }
    return out;
}

template <int D, bool F8, int MT, bool PG16>
struct Attend {
    // Positions a wave takes at once: 16 KB of keys and values in flight a wave
    // at 128 two-byte dims.  64 positions spill (MT = 4) or lose the second
    // wave of a SIMD: no faster anywhere.
    static constexpr int kTile = 32;
    static constexpr int kHalves = 2;  // of 16 positions
    static constexpr int kWaves = 4;
    static constexpr int kSteps = D / 32;   // products a 16-position score needs
    static constexpr int kKLoads = F8 ? D / 64 : D / 32;  // 16-byte loads of a key row's share
    static constexpr int kDpl = D / 16;     // dims a lane loads of a value row
    static constexpr int kVWords = F8 ? kDpl / 4 : kDpl / 2;
    static constexpr int kAcc = D / 4;      // accumulators a slot tile and lane
    // Weights are 2^(score - m) with m the running maximum plus kHold, so at most
    // 2^(8 - kHold), and m is raised by kRaise where a lane's sum has passed kFull.
    // A lane's 8 weights of a tile then add up to 2^-7, its sum stays below 2^-6 +
    // 2^-7, those of a slot's four lanes in four waves below 3/8 together: sums of
    // bf16 values stay in fp32's range however large the values are.  (Products
    // with values below 2^-108 are denormal, and weights below 2^-108 of the
    // largest are lost, below 2^-92 once m was raised, which takes a sum of 2^16
    // largest weights in a wave.)  e4m3 values, at most 448, need none of it.
    static constexpr float kHold = F8 ? 0.0f : 18.0f;
    static constexpr float kFull = 0x1p-6f, kRaise = 16.0f;
    static constexpr int kEsize = F8 ? 1 : 2;
    // waves a SIMD has registers for without spilling
    static constexpr int kOccupancy = D < 256 && MT * D <= 256 ? 2 : 1;

    union Smem {
        int lens[256];
        uint4 q[MT][kSteps][kWave];  // the queries as operand B, lane by lane
        // Partial results of slot tiles, lane by lane: running maximum (in
        // units of log2), sum and unnormalised output of slot lane % 16.
        struct {
            float acc[2][MT][kAcc / 4][kWave][4];
            float m[2][MT][kWave], l[2][MT][kWave];
        } part;
    };
};

// One of `blocks` workgroups of another kernel, over the positions behind a prefix.
template <int D, bool F8, int MT, bool PG16>
__device__ __forceinline__ void attend_own(const AttendArgs& a, unsigned block, unsigned blocks,
                                           typename Attend<D, F8, MT, PG16>::Smem& sm) {
    constexpr bool OWN = true;
#include "sv_attend_body.h"
}

}  // namespace
}  // namespace sv
