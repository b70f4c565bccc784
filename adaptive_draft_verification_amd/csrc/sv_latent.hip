// The paged cache of latent vectors (gfx950, wave64): sv_latent_append writes a
// step's vectors behind each request's context, sv_latent_attend lets the packed
// rows of every head attend to them.
#include "sv_attend.h"
#include "sv_device.h"
#include "sv_latent.h"
#include "sv_launch.h"

namespace sv {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// ------------------------------------------------------------------- append

// One thread per 16 bytes of new values.
template <bool F8>
__global__ void latent_append_kernel(LatentAppendArgs a) {
    const sv_latent_cache& c = a.cache;
    const int chunks = (c.latent_dim + SV_LATENT_ROPE) / 8;
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (int64_t)chunks * a.n_rows) return;
    const int row = (int)(i / chunks), d = (int)(i - (int64_t)row * chunks) * 8;
    const int r = a.row_req[row], j = a.row_pos[row];
    if (r == -1) return;
    if (r < 0 || r >= a.n_req || j < 0) {
        raise_error(a.dev_error, SV_DEV_BAD_CU_ROWS);
        return;
    }
    const int64_t t = (int64_t)a.ctx_len[r] + j;
    if (a.ctx_len[r] < 0 || t >= (int64_t)a.max_pages * c.page_size) {
        raise_error(a.dev_error, SV_DEV_BAD_CTX);
        return;
    }
    const int page = a.page_table[(int64_t)r * a.max_pages + (int)(t / c.page_size)];
    if (page < 0 || page >= c.n_pages) {
        raise_error(a.dev_error, SV_DEV_BAD_PAGE);
        return;
    }
    const uint16_t* src =
        d < c.latent_dim
            ? static_cast<const uint16_t*>(a.latent) + (int64_t)row * a.latent_ld + d
            : static_cast<const uint16_t*>(a.rope) + (int64_t)row * a.rope_ld + (d - c.latent_dim);
    const uint4 w = *reinterpret_cast<const uint4*>(src);
    const int64_t at =
        (int64_t)page * c.page_stride + (int64_t)(t % c.page_size) * c.token_stride + d;
    if (!F8) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(c.kv) + at) = w;
    } else {
        const float s = c.scale != nullptr ? *c.scale : 1.0f;
        *reinterpret_cast<int2*>(static_cast<uint8_t*>(c.kv) + at) = e4m3_of(w, s);
    }
}

// ------------------------------------------------------------------- attend
//
// A request's query slots are its rows times the heads (slot i: row i / H, head
// i % H): all of them read the same vectors.  A workgroup of four waves takes 32 WS
// slots over one part of the cached positions, N = 32 * 4 / WS of them at a time,
// in LDS as bf16; wave (ws, wp) takes 32 slots and 32 positions, with everything
// else in registers, in the operand layouts of v_mfma_f32_32x32x16_bf16:
//   S^T = K Q^T: operand A holds 32 positions (lane % 32) by 16 dims, B 32 slots by
//   the same dims, kept in registers over the whole length, so a lane ends with
//   scores of ONE slot (lane % 32) at positions 8 (i / 4) + 4 h + i % 4 (h = lane /
//   32, i = 0 .. 15);
//   O^T = C^T P^T: B's lane holds 8 positions of one slot, in the order in which
//   the lane has them from S; A needs the same 8 positions of one dim a lane:
//   two transposing LDS reads of 4 positions by 16 dims for each 16 lanes.
// With 32 slots a wave each KB read from LDS feeds 32 clocks of products: the
// 128 bytes a clock that LDS gives are two thirds used at full rate.  512 registers
// a lane: queries 4 (R + 64) / 16, accumulators R / 2.
// In LDS 8 positions by 8 chunks of 16 bytes are a KB, the chunk c of position x at
// (c ^ swizzle(x)) of its 128 bytes: 8 neighbouring positions' chunk c, and 4
// positions' chunks c and c ^ 1, lie in different banks.  A load brings one such KB,
// 8 lanes a position.

__device__ __forceinline__ int swizzle(int pos) { return ((pos & 3) << 1) | ((pos >> 2) & 1); }

template <int R, bool F8, int WS>
struct Latent {
    static constexpr int kWaves = 4, kWP = kWaves / WS, kTile = 32 * kWP;
    static constexpr int kDim = R + SV_LATENT_ROPE, kChunks = kDim / 8;
    static constexpr int kRow = kDim * 2;           // bytes
    static constexpr int kTileBytes = kTile * kRow;
    static constexpr int kGroups = kTile / 8 / kWaves;  // 8-position groups a wave brings
    static constexpr int kLoads = kChunks / 8;          // of each
    static constexpr int kGroup = kRow * 8;             // bytes
    static constexpr int kSteps = kDim / 16;        // products of a score
    static constexpr int kDims = R / 32;            // 32-dim tiles of the output
    static constexpr int kEsize = F8 ? 1 : 2;
    // Weights are 2^(score - m), m kHold above the first scores' maximum and raised
    // where a score passes that by 2^kSlack: weights are 2^-32 at most, so that sums
    // over 2^31 positions stay below 1 and sums of weighted values in fp32's range,
    // however large the values are.  Raising is rare: it takes the accumulators out
    // of the registers that products alone can use.
    static constexpr float kHold = 64.0f, kSlack = 32.0f;
};

template <int R, bool F8, int WS>
__global__ __launch_bounds__(256, 1) void latent_kernel(LatentAttendArgs a) {
    using C = Latent<R, F8, WS>;
    __shared__ __attribute__((aligned(16))) char tiles[2][C::kTileBytes];
    __shared__ int lens[256];
    __shared__ uint32_t absent[2][C::kWaves];  // bit i: position i of the wave's is none
    __shared__ uint32_t tainted[2][C::kWaves];
    const sv_latent_cache& c = a.cache;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 31, h = lane >> 5;
    const int ws = wave % WS, wp = wave / WS;
    // grid: slot blocks fastest, then requests and parts
    int id = spread(blockIdx.x, gridDim.x, a.slot_blocks);
    const int mb = id % a.slot_blocks;
    id /= a.slot_blocks;
    int r = id % a.n_req;
    const int part = id / a.n_req;
    if (a.longest_first) r = longest(r, a.ctx_len, a.n_req, lens);

    const int lo = a.cu_rows[r], hi = a.cu_rows[r + 1];
    const int rows = hi - lo;
    if (lo < 0 || hi < lo || rows > a.k_max + 1 || hi > a.q_rows) {
        if (threadIdx.x == 0) raise_error(a.dev_error, SV_DEV_BAD_CU_ROWS);
        return;
    }
    const int ctx = a.ctx_len[r];
    if (ctx < 0 || (int64_t)ctx + rows > (int64_t)a.max_pages * c.page_size) {
        if (threadIdx.x == 0) raise_error(a.dev_error, SV_DEV_BAD_CTX);
        return;
    }
    const int slots = rows * a.n_heads - mb * 32 * WS;  // slots of this block
    if (slots <= 0) return;
    const int len = ctx + rows;
    const int plen = part_len(len, a.parts, a.part_min);
    const int begin = part * plen, end = min(len, begin + plen);
    if (begin >= len) return;
    const bool whole = plen >= len;  // the request's only part

    // ---- the vectors' way into LDS: wave w brings the 8-position groups w kGroups ..
    const char* kv = static_cast<const char*>(c.kv);
    const int32_t* table = a.page_table + (int64_t)r * a.max_pages;
    const int mine = wave * C::kGroups * 8 + (lane >> 3);  // in the first group
    const int chunk_of = (lane & 7) ^ swizzle(lane >> 3);
    struct Pages {
        int id[C::kGroups];
    };
    auto pages_of = [&](int t0) {
        Pages p;
#pragma unroll
        for (int g = 0; g < C::kGroups; ++g) {
            const int t = min(t0 + mine + 8 * g, len - 1);
            p.id[g] = table[a.page_shift >= 0 ? t >> a.page_shift : t / c.page_size];
        }
        return p;
    };
    uint2 raw[F8 ? C::kGroups : 1][F8 ? C::kLoads : 1];
    bool bad = false;
    // issues the loads of the tile at t0, whose pages these are
    auto issue = [&](int t0, int buf, const Pages& pages) __attribute__((always_inline)) {
        uint32_t gone = 0;
#pragma unroll
        for (int g = 0; g < C::kGroups; ++g) {
            const int t = t0 + mine + 8 * g, page = pages.id[g];
            const int slot =
                t - (a.page_shift >= 0 ? t >> a.page_shift : t / c.page_size) * c.page_size;
            const bool there = t < end, good = page >= 0 && page < c.n_pages;
            bad |= there && !good;
            const char* from = kv + ((int64_t)page * c.page_stride + (int64_t)slot * c.token_stride +
                                     chunk_of * 8) *
                                        C::kEsize;
            char* to = tiles[buf] + (wave * C::kGroups + g) * C::kGroup;
            // bit i of a byte: the group's position i is none
            const uint64_t none = __ballot(!there || !good);
#pragma unroll
            for (int i = 0; i < 8; ++i) gone |= (uint32_t)((none >> (8 * i)) & 1) << (8 * g + i);
            if (there && good) {
#pragma unroll
                for (int i = 0; i < C::kLoads; ++i) {
                    if constexpr (F8) {
                        raw[g][i] = *reinterpret_cast<const uint2*>(from + i * 64);
                    } else {
                        __builtin_amdgcn_global_load_lds(
                            (const __attribute__((address_space(1))) void*)(from + i * 128),
                            (__attribute__((address_space(3))) void*)(to + i * 1024), 16, 0, 0);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < C::kLoads; ++i) {
                    if constexpr (F8) raw[g][i] = make_uint2(0, 0);
                    else *reinterpret_cast<uint4*>(to + i * 1024 + lane * 16) = make_uint4(0, 0, 0, 0);
                }
            }
        }
        if (lane == 0) absent[buf][wave] = gone;
    };
    // an 8-bit tile goes into LDS as bf16 when it has arrived
    auto settle = [&](int buf) __attribute__((always_inline)) {
        if constexpr (F8) {
#pragma unroll
            for (int g = 0; g < C::kGroups; ++g)
#pragma unroll
                for (int i = 0; i < C::kLoads; ++i) {
                    const uint2 v = raw[g][i];
                    char* to = tiles[buf] + (wave * C::kGroups + g) * C::kGroup + i * 1024 + lane * 16;
                    *reinterpret_cast<uint4*>(to) =
                        make_uint4(e4m3_pair<false>(v.x), e4m3_pair<true>(v.x),
                                   e4m3_pair<false>(v.y), e4m3_pair<true>(v.y));
                }
        }
    };

    int t0 = begin, buf = 0;
    issue(t0, 0, pages_of(t0));
    Pages pages = pages_of(t0 + C::kTile);

    // ---- queries of the wave's slots, operand B of every step
    const int slot = mb * 32 * WS + ws * 32 + col;
    const bool live = ws * 32 + col < slots;
    const int q_row = slot / a.n_heads, head = slot - q_row * a.n_heads;
    const int last = live ? ctx + q_row : -1;  // the last position the slot sees
    bf16x8 q[C::kSteps];
    {
        // a slot that is not there takes the first one's: it sees nothing
        const uint16_t* qp = static_cast<const uint16_t*>(a.q) +
                             (int64_t)(live ? lo + q_row : lo) * a.q_ld +
                             (int64_t)(live ? head : 0) * C::kDim + h * 8;
#pragma unroll
        for (int st = 0; st < C::kSteps; ++st) {
            const uint4 w = *reinterpret_cast<const uint4*>(qp + st * 16);
            q[st] = as_bf16x8(w.x, w.y, w.z, w.w);
        }
    }
    const float kv_scale = F8 && c.scale != nullptr ? *c.scale : 1.0f;
    const float scale = a.scale * kLog2e * kv_scale;

    f32x16 acc[C::kDims];
#pragma unroll
    for (int i = 0; i < C::kDims; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][e] = 0.0f;
    float m = -kInf, mu = 0.0f, l = 0.0f;  // running m (-inf: no score yet), the m used, sum

    // where a lane reads keys: chunks 2 st + h of its position
    const int k_pos = wp * 32 + col;
    const int k_at = (k_pos >> 3) * C::kGroup + (k_pos & 7) * 128;
    const int k_sw = swizzle(k_pos);
    // and values: 4 positions by 16 dims for 16 lanes
    const int v_pos = wp * 32 + 4 * h + ((lane & 15) >> 2);
    const int v_at = (v_pos >> 3) * C::kGroup + (v_pos & 7) * 128 + (lane & 1) * 8;
    const int v_sw = swizzle(v_pos);
    const int v_chunk = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);

    bool again = false;  // the tile at t0 is taken a second time, m having been raised
    for (;;) {
        float to = 0.0f;
        for (; t0 < end; t0 += C::kTile, buf ^= 1) {
            const bool edge = t0 + C::kTile > ctx;
            if (!again) {
                settle(buf);
                __builtin_amdgcn_s_waitcnt(0);
                __syncthreads();
                if (t0 + C::kTile < end) {
                    issue(t0 + C::kTile, buf ^ 1, pages);
                    pages = pages_of(t0 + 2 * C::kTile);
                }
                if (edge) {
                    // The step's own rows do not all see each other: a vector that is not
                    // finite may touch only those that see it.  It is zeroed, and its
                    // score is NaN.
                    uint32_t taint = 0;
                    for (int i = 0; i < C::kGroups * 8; ++i) {
                        const int pos = wave * C::kGroups * 8 + i;
                        if (t0 + pos <= ctx) continue;
                        uint4* at = reinterpret_cast<uint4*>(
                            tiles[buf] + (pos >> 3) * C::kGroup + (pos & 7) * 128 +
                            (lane >> 3) * 1024 + (lane & 7) * 16);
                        bool nf = false;
                        for (int ch = 0; ch < C::kChunks; ch += kWave) {
                            if (ch + lane >= C::kChunks) break;
                            const uint4 w = at[ch * 8];
                            nf |= bf16_pair_nonfinite(w.x) || bf16_pair_nonfinite(w.y) ||
                                  bf16_pair_nonfinite(w.z) || bf16_pair_nonfinite(w.w);
                        }
                        if (__ballot(nf) == 0) continue;
                        taint |= 1u << i;
                        for (int ch = 0; ch < C::kChunks; ch += kWave)
                            if (ch + lane < C::kChunks) at[ch * 8] = make_uint4(0, 0, 0, 0);
                    }
                    if (lane == 0) tainted[buf][wave] = taint;
                    __syncthreads();
                }
            }
            const char* tile = tiles[buf];
            uint64_t none = 0, nan = 0;  // positions of the tile
#pragma unroll
            for (int w = 0; w < C::kWaves; ++w) {
                none |= (uint64_t)absent[buf][w] << (w * C::kGroups * 8);
                if (edge) nan |= (uint64_t)tainted[buf][w] << (w * C::kGroups * 8);
            }
            const uint32_t no = (uint32_t)(none >> (wp * 32)), nn = (uint32_t)(nan >> (wp * 32));

            // LDS reads stay kAhead products ahead of their own, in this order
            constexpr int kAhead = 4;
            auto key = [&](int st) __attribute__((always_inline)) {
                const int chunk = 2 * st + h;
                const uint4 w = *reinterpret_cast<const uint4*>(
                    tile + k_at + (st >> 2) * 1024 + ((chunk & 7) ^ k_sw) * 16);
                return as_bf16x8(w.x, w.y, w.z, w.w);
            };
            f32x16 s;
#pragma unroll
            for (int e = 0; e < 16; ++e) s[e] = 0.0f;
            bf16x8 k8[kAhead];
#pragma unroll
            for (int st = 0; st < kAhead; ++st) k8[st] = key(st);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int st = 0; st < C::kSteps; ++st) {
                s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k8[st % kAhead], q[st], s, 0, 0, 0);
                if (st + kAhead < C::kSteps) k8[st % kAhead] = key(st + kAhead);
                __builtin_amdgcn_sched_barrier(0);
            }

            float p[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) p[e] = s[e] * scale;
            if (edge || (no | nn) != 0) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int pos = 8 * (e >> 2) + 4 * h + (e & 3);
                    if ((nn >> pos) & 1) p[e] = __builtin_nanf("");
                    if (((no >> pos) & 1) || t0 + wp * 32 + pos > last) p[e] = -kInf;
                }
            }
            float mx = p[0];
#pragma unroll
            for (int e = 1; e < 16; ++e) mx = fmaxf(mx, p[e]);
            if (__ballot(mx > m + (C::kSlack - C::kHold)) != 0) {
                mx = fmaxf(mx, __shfl_xor(mx, 32));
                to = fmaxf(m, mx + C::kHold);
                // the slot's first scores: nothing to rescale yet
                if (m == -kInf && to > m) m = mu = to;
                if (__ballot(to > m + C::kSlack) != 0) break;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                p[e] = fast_exp2(p[e] - mu);
                l += p[e];
            }
            // Weights go into the product as two bf16 terms, the upper half of the fp32
            // weight and the rest, off by at most 2^-15 of each: one term's 2^-8 would
            // show in the result beside its own rounding.  Both are positive where the
            // weight is (the rest of 1 + 2^-23 times it is taken): an infinite value
            // times 0 or a negative rest would make NaN.
            constexpr float kOneUp = 1.0f + 0x1p-23f;
            bf16x8 pb[2], pr[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                uint32_t hw[4], rw[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = p[8 * t + 2 * i], y = p[8 * t + 2 * i + 1];
                    const uint32_t xb = __float_as_uint(x), yb = __float_as_uint(y);
                    hw[i] = __builtin_amdgcn_perm(yb, xb, 0x07060302u);
                    rw[i] = pack_bf16(fmaf(x, kOneUp, -bf16_hi(xb)), fmaf(y, kOneUp, -bf16_hi(yb)));
                }
                pb[t] = as_bf16x8(hw[0], hw[1], hw[2], hw[3]);
                pr[t] = as_bf16x8(rw[0], rw[1], rw[2], rw[3]);
            }
            // 16 positions (half t of the wave's) of 32 dims
            auto value = [&](int it) __attribute__((always_inline)) {
                const int i = it >> 1, t = it & 1;
                const int chunk = 4 * i + v_chunk;
                const char* at = tile + v_at + t * 2 * C::kGroup + (i >> 1) * 1024 +
                                 ((chunk & 7) ^ v_sw) * 16;
                const s16x4 x0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4*)at);
                const s16x4 x1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4*)(at + C::kGroup));
                uint2 w0, w1;
                __builtin_memcpy(&w0, &x0, 8);
                __builtin_memcpy(&w1, &x1, 8);
                return as_bf16x8(w0.x, w0.y, w1.x, w1.y);
            };
            bf16x8 v8[kAhead];
#pragma unroll
            for (int it = 0; it < kAhead; ++it) v8[it] = value(it);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int it = 0; it < 2 * C::kDims; ++it) {
                const int i = it >> 1, t = it & 1;
                acc[i] =
                    __builtin_amdgcn_mfma_f32_32x32x16_bf16(v8[it % kAhead], pb[t], acc[i], 0, 0, 0);
                acc[i] =
                    __builtin_amdgcn_mfma_f32_32x32x16_bf16(v8[it % kAhead], pr[t], acc[i], 0, 0, 0);
                if (it + kAhead < 2 * C::kDims) v8[it % kAhead] = value(it + kAhead);
                __builtin_amdgcn_sched_barrier(0);
            }
            again = false;
        }
        if (t0 >= end) break;
        const float f = to > m ? fast_exp2(m - to) : 1.0f;
        if (to > m) {
            l *= f;
            m = mu = to;
        }
#pragma unroll
        for (int i = 0; i < C::kDims; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][e] *= f;
        again = true;
    }
    if (__ballot(bad) != 0 && lane == 0) raise_error(a.dev_error, SV_DEV_BAD_PAGE);

    // the other half's positions of the slot
    l += __shfl_xor(l, 32);
    if constexpr (C::kWP == 2) {
        // and the other wave's: its accumulators, lane by lane, through LDS
        __syncthreads();
        f32x4* give = reinterpret_cast<f32x4*>(tiles[0]) + ws * (C::kDims * 4 + 1) * kWave + lane;
        static_assert(WS * (C::kDims * 4 + 1) * kWave * 16 <= 2 * C::kTileBytes, "fits in the tiles");
        if (wp == 1) {
#pragma unroll
            for (int i = 0; i < C::kDims; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    give[(i * 4 + e) * kWave] = f32x4{acc[i][4 * e], acc[i][4 * e + 1],
                                                      acc[i][4 * e + 2], acc[i][4 * e + 3]};
            give[C::kDims * 4 * kWave] = f32x4{m, l, 0.0f, 0.0f};
        }
        __syncthreads();
        if (wp == 1) return;
        const f32x4 ml = give[C::kDims * 4 * kWave];
        const float mx = fmaxf(m, ml[0]);
        const float f1 = m == mx ? 1.0f : fast_exp2(m - mx);
        const float f2 = ml[0] == mx ? 1.0f : fast_exp2(ml[0] - mx);
        l = l * f1 + ml[1] * f2;
        m = mx;
#pragma unroll
        for (int i = 0; i < C::kDims; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f32x4 o = give[(i * 4 + e) * kWave];
#pragma unroll
                for (int x = 0; x < 4; ++x) acc[i][4 * e + x] = acc[i][4 * e + x] * f1 + o[x] * f2;
            }
    }
    if (!whole) {
        if (!live) return;
        const int64_t rec =
            (((int64_t)r * (a.k_max + 1) + q_row) * a.n_heads + head) * a.parts + part;
        float* o = a.part_out + rec * R + 4 * h;
#pragma unroll
        for (int i = 0; i < C::kDims; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *reinterpret_cast<f32x4*>(o + i * 32 + e * 8) = f32x4{
                    acc[i][4 * e], acc[i][4 * e + 1], acc[i][4 * e + 2], acc[i][4 * e + 3]};
        if (h == 0) {
            a.part_ml[rec * 2] = m;
            a.part_ml[rec * 2 + 1] = l;
        }
        return;
    }
    // no weight at all: 0, also where 0 times a value was NaN
    const bool nothing = l == 0.0f;
    const float inv = nothing ? 0.0f : 1.0f / l;
    uint16_t* o = static_cast<uint16_t*>(a.out) + (int64_t)(lo + q_row) * a.out_ld +
                  (int64_t)head * R + 8 * h;
#pragma unroll
    for (int i = 0; i < C::kDims; ++i)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            // dims 16 g .. 16 g + 7 and + 8 .. + 15 of the tile: halves of both in either
            // half of the wave, exchanged so that a lane stores 8 in a row
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = acc[i][8 * g + 2 * e], y = acc[i][8 * g + 2 * e + 1];
                // the mean first, then its scale: only their product has to be in range
                w[e] = nothing ? 0u : pack_bf16(x * inv * kv_scale, y * inv * kv_scale);
            }
            const auto s0 = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
            const auto s1 = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
            if (live)
                *reinterpret_cast<uint4*>(o + i * 32 + g * 16) =
                    make_uint4(s0[0], s1[0], s0[1], s1[1]);
        }
    if (live && a.out_lse != nullptr && h == 0)
        a.out_lse[(int64_t)(lo + q_row) * a.n_heads + head] =
            nothing ? -kInf : ((m - C::kHold) + log2f(l * exp2f(C::kHold))) * kLn2;
}

// Merges the parts of a (row, head), a wave each: lanes over the dims.
template <int R, bool F8>
__global__ __launch_bounds__(256) void latent_join_kernel(LatentAttendArgs a) {
    constexpr int E = R / kWave;
    constexpr float kHold = Latent<R, F8, 2>::kHold;
    __shared__ float factors[4][128];
    const sv_latent_cache& c = a.cache;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int per = (a.k_max + 1) * a.n_heads;
    const int64_t id = (int64_t)blockIdx.x * 4 + wave;
    if (id >= (int64_t)a.n_req * per) return;
    const int r = (int)(id / per), rest = (int)(id % per);
    const int row = rest / a.n_heads, head = rest % a.n_heads;
    const int lo = a.cu_rows[r], hi = a.cu_rows[r + 1], rows = hi - lo, ctx = a.ctx_len[r];
    if (lo < 0 || hi < lo || rows > a.k_max + 1 || hi > a.q_rows || row >= rows || ctx < 0 ||
        (int64_t)ctx + rows > (int64_t)a.max_pages * c.page_size)
        return;
    const int len = ctx + rows, plen = part_len(len, a.parts, a.part_min);
    if (plen >= len) return;
    const int n = (len + plen - 1) / plen;  // at most 128
    const int64_t rec = id * a.parts;
    const float* ml = a.part_ml + rec * 2;
    const float* po = a.part_out + rec * R + lane * E;
    // the largest maximum and the parts' factors, two a lane
    float m0 = -kInf, m1 = -kInf, l0 = 0.0f, l1 = 0.0f;
    if (lane < n) m0 = ml[2 * lane], l0 = ml[2 * lane + 1];
    if (lane + 64 < n) m1 = ml[2 * lane + 128], l1 = ml[2 * lane + 129];
    const float m = wave_max(fmaxf(m0, m1));
    const float f0 = m0 == m ? 1.0f : fast_exp2(m0 - m);
    const float f1 = m1 == m ? 1.0f : fast_exp2(m1 - m);
    const float l = wave_sum((lane < n ? f0 * l0 : 0.0f) + (lane + 64 < n ? f1 * l1 : 0.0f));
    // over the whole sum before the outputs are added up: they are then shares of the
    // mean, and stay in range
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    float* factor = factors[wave];
    factor[lane] = f0 * inv;
    factor[lane + 64] = f1 * inv;
    __builtin_amdgcn_wave_barrier();
    float o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
    for (int p0 = 0; p0 < n; p0 += 4) {
        float x[4][E];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) x[i][e] = po[(int64_t)min(p0 + i, n - 1) * R + e];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (p0 + i >= n) break;
            const float f = factor[p0 + i];
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] += f * x[i][e];
        }
    }
    const float kv_scale = F8 && c.scale != nullptr ? *c.scale : 1.0f;
    uint32_t w[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2)
        w[e / 2] = l == 0.0f ? 0u : pack_bf16(o[e] * kv_scale, o[e + 1] * kv_scale);
    __builtin_memcpy(static_cast<uint16_t*>(a.out) + (int64_t)(lo + row) * a.out_ld +
                         (int64_t)head * R + lane * E,
                     w, sizeof(w));
    if (a.out_lse != nullptr && lane == 0)
        a.out_lse[(int64_t)(lo + row) * a.n_heads + head] =
            l == 0.0f ? -kInf : ((m - kHold) + log2f(l * exp2f(kHold))) * kLn2;
}

template <int R, bool F8>
hipError_t run_latent(const LatentAttendArgs& a, hipStream_t stream) {
    const unsigned grid = (unsigned)((int64_t)a.n_req * a.slot_blocks * a.parts);
    if (a.slot_waves == 4) latent_kernel<R, F8, 4><<<grid, 256, 0, stream>>>(a);
    else latent_kernel<R, F8, 2><<<grid, 256, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.parts == 1) return e;
    const int64_t total = (int64_t)a.n_req * (a.k_max + 1) * a.n_heads;
    latent_join_kernel<R, F8><<<(unsigned)((total + 3) / 4), 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_latent_append(const LatentAppendArgs& a, hipStream_t stream) {
    const int64_t threads = (int64_t)a.n_rows * ((a.cache.latent_dim + SV_LATENT_ROPE) / 8);
    const unsigned grid = (unsigned)((threads + 255) / 256);
    if (a.cache.dtype == SV_E4M3) latent_append_kernel<true><<<grid, 256, 0, stream>>>(a);
    else latent_append_kernel<false><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_latent_attend(const LatentAttendArgs& a, hipStream_t stream) {
    const bool f8 = a.cache.dtype == SV_E4M3;
    if (a.cache.latent_dim == 512)
        return f8 ? run_latent<512, true>(a, stream) : run_latent<512, false>(a, stream);
    return f8 ? run_latent<256, true>(a, stream) : run_latent<256, false>(a, stream);
}

}  // namespace sv
