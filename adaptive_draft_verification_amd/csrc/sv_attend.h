// Device-side helpers shared by the attention kernels (gfx950, wave64).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sv_device.h"

namespace sv {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_inff();

__device__ __forceinline__ bf16x8 as_bf16x8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t w[4] = {a, b, c, d};
    bf16x8 r;
    __builtin_memcpy(&r, w, 16);
    return r;
}

// Two e4m3 values (low or high half of w) as two bf16: exact.
template <bool HI>
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w) {
    const bf16x2 v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI);
    uint32_t r;
    __builtin_memcpy(&r, &v, 4);
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const f32x2 f = {a, b};
    const bf16x2 v = __builtin_convertvector(f, bf16x2);
    uint32_t r;
    __builtin_memcpy(&r, &v, 4);
    return r;
}

__device__ __forceinline__ bool bf16_pair_nonfinite(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// Eight bf16 values over s as e4m3: x / s rounded to fp32, then to the nearest
// (ties to even), held at the type's largest value; NaN stays NaN.
__device__ __forceinline__ int2 e4m3_of(const uint4& w, float s) {
    float x[8] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y),
                  bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w)};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x[e] = __fdiv_rn(x[e], s);
        x[e] = x[e] > 448.0f ? 448.0f : x[e] < -448.0f ? -448.0f : x[e];
    }
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], hi, true);
    return make_int2(lo, hi);
}

// 8 bytes of device memory: a pointer kept in LDS does not tell the compiler that it is
// one, and a load that may be of LDS waits for that too.
__device__ __forceinline__ uint2 load_global8(const char* p) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 w = *(const __attribute__((address_space(1))) u32x2*)p;
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

// 16 bytes a lane from `from` + i STEP (each lane's own) to LDS at `to` + 16 lane (the
// same `to` in every lane), without registers.  Done when vmcnt says so: the
// caller waits, then meets the other waves at a barrier.  In assembly because
// the compiler waits for such a load before any later read of LDS, whichever
// part of it that reads.  The instruction's offset counts in both addresses.
template <int STEP>
__device__ __forceinline__ void load_to_lds(const char* from, uint32_t to, int i) {
    uint32_t keep;  // m0 is the compiler's
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
                 "global_load_lds_dwordx4 %2, off offset:%3\n\ts_mov_b32 m0, %0"
                 : "=&s"(keep)
                 : "s"(__builtin_amdgcn_readfirstlane(to - i * STEP)), "v"(from), "i"(i * STEP)
                 : "memory");
}

// The request of rank `rank` by context length, longest first (ties to the
// lower request): where workgroups take turns on the CUs, a long request that
// starts last would be waited for alone (256 requests of 0 .. 4096 positions: 429
// us in their own order, 394 this way).  For up to 256 requests, a thread each;
// more keep their own order (256 requests 393 us, 257 424).
__device__ __forceinline__ int longest(int rank, const int32_t* ctx_len, int n, int* lens) {
    __shared__ int found;
    const int t = threadIdx.x;
    // lengths from 2^22 on count as equal: any order is a right one
    const int mine = t < n ? (min(max(ctx_len[t], 0), (1 << 22) - 1) << 8) | (255 - t) : -1;
    lens[t] = mine;
    __syncthreads();
    int ahead = 0;
#pragma unroll 4
    for (int j = 0; j < n; j += 4) {
        const int4 v = *reinterpret_cast<const int4*>(lens + j);
        ahead += (v.x > mine) + (v.y > mine) + (v.z > mine) + (v.w > mine);
    }
    if (t < n && ahead == rank) found = t;
    __syncthreads();
    return found;
}

// Consecutive workgroups go to the eight XCDs in turn, each with an L2 of its
// own; `run` neighbouring work items that read the same lines (slot blocks of
// a head, heads narrower than a line) are given to one XCD, one behind the
// other: 64 requests, 16 heads of 64 bytes: 42 us without, 29 with.
__device__ __forceinline__ int spread(int b, int total, int run) {
    const int group = 8 * run, g = b / group, rest = b - g * group;
    if ((g + 1) * group > total) return b;
    return g * group + (rest & 7) * run + (rest >> 3);
}

}  // namespace
}  // namespace sv
