// Attention of a batch whose requests share prefixes (gfx950, wave64):
// sv_cache_attend_shared.  Three launches: the groups laid out; every group's rows over
// its prefix, as one long block of queries, and every request's rows over its own
// positions (sv_cache_attend's kernel, from the prefix's end on); the join.
#include <type_traits>

#include "sv_attend_kernel.h"
#include "sv_device.h"
#include "sv_launch.h"
#include "sv_shared.h"

namespace sv {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// ------------------------------------------------------------------- layout

__device__ __forceinline__ int64_t wave_incl_sum64(int64_t v, int lane) {
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const int64_t x = __shfl_up((long long)v, off);
        if (lane >= off) v += x;
    }
    return v;
}

// Checks the groups and their requests, and counts the tiles: one workgroup, so that
// the launches behind it only read.  KEEP: at most T requests; what is read more than
// once is kept in LDS then, and one round trip to memory is left of six (2 requests
// 5.2 -> 3.6 us).
template <int T, bool KEEP>
__global__ __launch_bounds__(T) void layout_kernel(SharedArgs s) {
    const AttendArgs& a = s.own;
    constexpr int kKeep = KEEP ? T : 1;
    __shared__ int kept_start[kKeep + 1], kept_prefix[kKeep], kept_cu[kKeep + 1];
    __shared__ int kept_broken[kKeep];
    __shared__ int block_sums[T / kWave], longest_prefix;
    __shared__ int64_t tile_sums[T / kWave];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    if (t == 0) longest_prefix = 0;
    if (KEEP) {
        for (int i = t; i <= a.n_req; i += T) kept_cu[i] = a.cu_rows[i];
        if (s.n_groups > 0)
            for (int i = t; i <= s.n_groups; i += T) kept_start[i] = s.group_start[i];
        if (t < s.n_groups) kept_prefix[t] = s.prefix_len[t];
        __syncthreads();
    }
    auto start = [&](int g) { return KEEP ? kept_start[g] : s.group_start[g]; };
    auto prefix_of = [&](int g) { return KEEP ? kept_prefix[g] : s.prefix_len[g]; };
    auto cu = [&](int r) { return KEEP ? kept_cu[r] : a.cu_rows[r]; };
    auto broken = [&](int g) -> int* { return KEEP ? kept_broken + g : &s.group[g].broken; };
    auto bits_of = [&](int g) {
        return KEEP ? kept_broken[g]
                    : __hip_atomic_load(&s.group[g].broken, __ATOMIC_RELAXED,
                                        __HIP_MEMORY_SCOPE_AGENT);
    };
    int err = 0;
    for (int g = t; g <= s.n_groups && s.n_groups > 0; g += T) {
        const int at = start(g);
        if (at < 0 || at > a.n_req || (g > 0 && start(g - 1) > at)) err = SV_DEV_BAD_CU_ROWS;
    }
    for (int g = t; g < s.n_groups; g += T) {
        const int P = prefix_of(g);
        const bool fits = P >= 0 && P <= (int64_t)a.max_pages * a.cache.page_size;
        if (KEEP)
            kept_broken[g] = fits ? 0 : SV_DEV_BAD_CTX;
        else
            __hip_atomic_store(&s.group[g].broken, fits ? 0 : SV_DEV_BAD_CTX, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
    }
    const bool none = __syncthreads_or(err) != 0;
    // every request's group, and whether its rows are where they have to be
    int group = -1;  // of the thread's request (KEEP)
    for (int r = t; r < a.n_req; r += T) {
        group = -1;
        if (!none && s.n_groups > 0 && r >= start(0) && r < start(s.n_groups)) {
            int lo = 0, hi = s.n_groups;  // the last group that starts at r or before
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (start(mid) <= r) lo = mid;
                else hi = mid;
            }
            group = lo;
            const int from = cu(r), to = cu(r + 1);
            if (from < 0 || to < from || to - from > a.k_max + 1 || to > a.q_rows)
                atomicOr(broken(group), SV_DEV_BAD_CU_ROWS);
        }
        if (!KEEP) s.request[r].group = group;
    }
    __syncthreads();
    int blocks = 0;  // of earlier groups
    int64_t tiles = 0;
    for (int g0 = 0; g0 < s.n_groups; g0 += T) {
        const int g = g0 + t;
        int n = 0, each = 0;
        if (g < s.n_groups && !none) {
            const int bits = bits_of(g);
            err |= bits;
            const int from = start(g), to = start(g + 1), P = prefix_of(g);
            if (bits == 0 && P > 0 && to > from)
                n = ((cu(to) - cu(from)) * a.group + SharedPlan::kSlots - 1) / SharedPlan::kSlots;
            if (n > 0) {
                each = (int)(((int64_t)P + SharedPlan::kTile - 1) / SharedPlan::kTile);
                atomicMax(&longest_prefix, each);
            }
        }
        const int blocks_to = wave_incl_sum_dpp(n, lane);
        const int64_t tiles_to = wave_incl_sum64((int64_t)n * each, lane);
        if (lane == 63) {
            block_sums[wave] = blocks_to;
            tile_sums[wave] = tiles_to;
        }
        __syncthreads();
        int block = blocks + blocks_to - n;
        int64_t tile = tiles + tiles_to - (int64_t)n * each;
        for (int w = 0; w < T / kWave; ++w) {
            if (w < wave) {
                block += block_sums[w];
                tile += tile_sums[w];
            }
            blocks += block_sums[w];
            tiles += tile_sums[w];
        }
        if (g < s.n_groups) {
            s.group[g].tile = tile;
            s.group[g].block = block;
        }
        __syncthreads();
    }
    if (t == 0) {
        s.group[s.n_groups].tile = tiles;
        s.group[s.n_groups].block = blocks;
        // equal runs; a block of n tiles lies in n / run + 2 of them at most
        const int64_t all = tiles * a.cache.n_kv_heads;
        const int64_t few =
            (longest_prefix + SharedPlan::kSegments - 3) / (SharedPlan::kSegments - 2);
        int64_t run = s.chunks > 0 ? (all + s.chunks - 1) / s.chunks : 0;
        run = run < few ? few : run;
        run = run < SharedPlan::kRunMin ? SharedPlan::kRunMin : run;
        s.totals->run = run;
        s.totals->chunks = (int)((all + run - 1) / run);
    }
    for (int r = t; r < a.n_req; r += T) {
        const int g = KEEP ? group : s.request[r].group;
        int first = none ? -1 : 0, row = 0;
        if (g >= 0) {
            first = bits_of(g) != 0 ? -1 : prefix_of(g);
            row = cu(r) - cu(start(g));
        }
        s.first[r] = first;
        s.request[r] = SharedRequest{g, row};
    }
    if (err != 0) raise_error(a.dev_error, err);
}

// ------------------------------------------------------------------- prefix
//
// A group's query slots of one kv head are its rows times the G query heads that
// share it (slot i: row i / G, head h G + i % G): all of them see the whole prefix.
// A workgroup of four waves takes 128 slots over a run of tiles of 32 positions, whose
// keys and values lie in LDS as bf16; a wave takes 32 slots.  Operands of
// v_mfma_f32_32x32x16_bf16:
//   S^T = K Q^T: A holds 32 positions (lane % 32) by 16 dims (8 for each g = lane / 32),
//   B 32 slots by the same dims, so a lane ends with 16 scores of ONE slot (lane % 32),
//   at positions 4 g .. 4 g + 3 of each 8;
//   O^T = V^T P^T: B's lane holds 8 positions of its slot, 4 g .. of two eights, just as
//   the scores are; A needs the same positions of one dim (lane % 32): two transposing
//   LDS reads of 4 positions by 16 dims for each 16 lanes.
// What bounds it: at 128 dims 24 products of 32 clocks a wave and tile, and on the same
// issue port some 105 other instructions of 4 clocks (exp2 8), beside which a product
// takes 8 (measured; one of 16 x 16 x 32, of half the work, as many).  A tile takes a
// wave 1950 clocks alone on its SIMD and two waves 2400: scores 280, their maxima 180,
// products with the values 690, the rest waits for LDS, for the other waves and for the
// loads' issue.  Other orders of the same instructions all came out within 3 %.
// In LDS 8 positions by 8 chunks of 16 bytes are a KB, the chunk c of position x at
// (c ^ swizzle(x)) of its 128 bytes.  LDS has 64 banks of 4 bytes: the chunk c of 16
// neighbouring positions, and the chunks c and c ^ 1 of 8, lie in different ones.

__device__ __forceinline__ int swizzle(int pos) { return (pos & 6) | ((pos >> 3) & 1); }

// What a position without a page is loaded from.
__device__ const uint4 kZeros[256 / 8] = {};

template <int D, bool F8>
struct Prefix {
    static constexpr int kTile = SharedPlan::kTile;
    static constexpr int kLoads = D / 64;           // KB of 8 positions' keys, or values
    static constexpr int kGroup = kLoads * 1024;    // bytes
    static constexpr int kBytes = 4 * kGroup;       // of a tile's keys, or values: a group a wave
    static constexpr int kSteps = D / 16;           // products of a score
    static constexpr int kDims = D / 32;            // 32-dim tiles of the output
    static constexpr int kEsize = F8 ? 1 : 2;
    static constexpr int kPlaces = 512;             // positions whose places are in LDS
    static constexpr int kOccupancy = D < 256 ? 2 : 1;
    // Weights are held as attend_kernel holds them: 2^(score - m), m kHold above the
    // maximum that it was set from, raised where a score passes that by 2^8 or a lane's
    // sum kFull.
    static constexpr float kHold = F8 ? 0.0f : 18.0f, kSlack = 8.0f;
    static constexpr float kFull = 0x1p-6f, kRaise = 16.0f;

    struct Smem {
        __attribute__((aligned(16))) char keys[3][kBytes];
        __attribute__((aligned(16))) char values[4][kBytes];
        // of position begin + i at i % kPlaces: where its key and its value are, and
        // whether there is none
        const char* key_at[kPlaces];
        const char* value_at[kPlaces];
        __attribute__((aligned(4))) uint8_t absent[kPlaces];
        int holes;  // a position before the end is none
    };
};

// Workgroup `id` of s.chunks.
template <int D, bool F8>
__device__ __forceinline__ void prefix(const SharedArgs& s, int id,
                                       typename Prefix<D, F8>::Smem& sm) {
    using C = Prefix<D, F8>;
    const AttendArgs& a = s.own;
    const sv_cache& c = a.cache;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 31, g = lane >> 5;
    // consecutive runs of tiles (they read the same keys and values) to one XCD: every
    // eighth workgroup
    const SharedTotals totals = *s.totals;
    const int each = (totals.chunks + 7) / 8;
    const int chunk = (id % 8) * each + id / 8;
    if (id / 8 >= each || chunk >= totals.chunks) return;
    const int64_t head_tiles = s.group[s.n_groups].tile;
    const int head_blocks = s.group[s.n_groups].block;
    int64_t tile = chunk * totals.run;
    const int64_t to_tile = min(tile + totals.run, head_tiles * c.n_kv_heads);
    int h = (int)(tile / head_tiles);
    int64_t in_head = tile - h * head_tiles;
    // the group the run starts in: the last one whose tiles begin there or before
    int group = 0;
    for (int n = s.n_groups; n > 1;) {
        const int step = (n + kWave - 1) / kWave, at = group + lane * step;
        const bool before = lane * step < n && s.group[at].tile <= in_head;
        const int skip = (__popcll(__ballot(before)) - 1) * step;  // lane 0's is
        group += skip;
        n = min(step, n - skip);
    }
    // where a lane reads keys: chunk 2 st + g of its position, st = 0 .. 3 of 128 bytes;
    // and values: 4 positions by 16 dims for 16 lanes, in the first or second 8 positions,
    // of either 32 dims
    int k_at[4], v_at[2][2];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        k_at[j] = (col >> 3) * C::kGroup + (col & 7) * 128 + ((2 * j + g) ^ swizzle(col)) * 16;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int pos = 8 * r + 4 * g + ((lane & 15) >> 2);
            const int ch = 4 * j + 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
            v_at[r][j] = (pos >> 3) * C::kGroup + (pos & 7) * 128 + (lane & 1) * 8 +
                         (ch ^ swizzle(pos)) * 16;
        }
    // keys' and values' way into LDS: wave w brings positions 8 w .. of a tile
    const int mine = wave * 8 + (lane >> 3);
    const int chunk_of = ((lane & 7) ^ swizzle(mine)) * 8 * C::kEsize;
    bool bad = false;
    if (threadIdx.x == 0) sm.holes = 0;

    // ---- the run's segments
    while (tile < to_tile) {
        if (in_head == head_tiles) {
            in_head = 0;
            group = 0;
            ++h;
        }
        while (s.group[group + 1].tile <= in_head) ++group;
        const int from_req = s.group_start[group], to_req = s.group_start[group + 1];
        const int P = s.prefix_len[group];
        const int lo = a.cu_rows[from_req];
        const int block_tiles = (int)(((int64_t)P + C::kTile - 1) / C::kTile);
        const int64_t in_group = in_head - s.group[group].tile;
        const int index = (int)((uint64_t)in_group / (uint32_t)block_tiles);  // the block's
        const int first_tile = (int)(in_group - (int64_t)index * block_tiles);
        const int n_tiles = (int)min((int64_t)(block_tiles - first_tile), to_tile - tile);
        const int64_t block_id = (int64_t)h * head_blocks + s.group[group].block + index;
        const int slots = (a.cu_rows[to_req] - lo) * a.group - index * SharedPlan::kSlots;
        const int begin = first_tile * C::kTile;
        const int end = min(P, begin + n_tiles * C::kTile);
        if (threadIdx.x == 0) {
            if (first_tile == 0) s.span[block_id].first = chunk;
            if (first_tile + n_tiles == block_tiles) s.span[block_id].last = chunk;
        }
        tile += n_tiles;
        in_head += n_tiles;

        // The places of `n` positions from `from` on, into LDS: kPlaces at first, then
        // half as many at a time (a wait for a page id in registers would be a wait for
        // the tiles that are on their way).  None: after the end, or on a page that is
        // not there.
        const int32_t* table = a.page_table + (int64_t)from_req * a.max_pages;
        const int64_t of_head = (int64_t)h * c.head_stride * C::kEsize;
        const char* k_base = static_cast<const char*>(c.k) + of_head;
        const char* v_base = static_cast<const char*>(c.v) + of_head;
        auto fetch_places = [&](int from, int n) __attribute__((always_inline)) {
            for (int i = threadIdx.x; i < n; i += 256) {
                // (positions past the last ones looked up are not reached: no overflow)
                const int64_t t = (int64_t)from + i;
                const char *k = reinterpret_cast<const char*>(kZeros), *v = k;
                bool none = true;
                if (t < end) {
                    const int in = a.page_shift >= 0
                                       ? (int)t >> a.page_shift
                                       : (int)((unsigned)t / (unsigned)c.page_size);
                    const int page = table[in];
                    if (page >= 0 && page < c.n_pages) {
                        const int64_t place =
                            ((int64_t)page * c.page_stride +
                             (int64_t)((int)t - in * c.page_size) * c.token_stride) *
                            C::kEsize;
                        k = k_base + place;
                        v = v_base + place;
                        none = false;
                    } else {
                        bad = true;
                        sm.holes = 1;
                    }
                }
                const int at = (int)(t - begin) & (C::kPlaces - 1);
                sm.key_at[at] = k;
                sm.value_at[at] = v;
                sm.absent[at] = none;
            }
        };
        auto place = [&](int t) __attribute__((always_inline)) {  // of the lane's in tile t
            return (t * C::kTile + mine) & (C::kPlaces - 1);
        };
        uint2 raw[F8 ? 2 * C::kLoads : 1];
        // issues load i of a tile's keys, or of its values
        auto bring = [&](const char* from, char* into, int keys, int i)
                         __attribute__((always_inline)) {
            from += chunk_of;
            if constexpr (F8) {
                raw[(keys ? 0 : C::kLoads) + i] = load_global8(from + i * 64);
            } else {
                const uint32_t to =
                    __builtin_amdgcn_readfirstlane(lds_address(into + wave * C::kGroup));
                load_to_lds<128>(from, to + i * 1024, i);
            }
        };
        auto bring_all = [&](const char* from, char* into, int keys)
                             __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < C::kLoads; ++i) bring(from, into, keys, i);
        };
        // 8-bit ones pass registers and go into LDS as bf16
        auto widen = [&](char* into, int keys) __attribute__((always_inline)) {
            if constexpr (F8) {
#pragma unroll
                for (int i = 0; i < C::kLoads; ++i) {
                    const uint2 w = raw[(keys ? 0 : C::kLoads) + i];
                    *reinterpret_cast<uint4*>(into + wave * C::kGroup + i * 1024 + lane * 16) =
                        make_uint4(e4m3_pair<false>(w.x), e4m3_pair<true>(w.x),
                                   e4m3_pair<false>(w.y), e4m3_pair<true>(w.y));
                }
            }
        };

        __syncthreads();  // the segment before has been read
        fetch_places(begin, C::kPlaces);
        __syncthreads();
        // bf16: the keys of tiles 0 .. 2 and the values of 0 and 1; 8 bits: the keys of 0
        bring_all(sm.key_at[place(0)], sm.keys[0], 1);
        if (!F8) {
#pragma unroll
            for (int t = 1; t < 3; ++t) {
                bring_all(sm.key_at[place(t)], sm.keys[t], 1);
                bring_all(sm.value_at[place(t - 1)], sm.values[t - 1], 0);
            }
        }

        // ---- queries of the wave's slots, operand B of every step
        const int slot = index * SharedPlan::kSlots + wave * 32 + col;
        const bool live = wave * 32 + col < slots;
        bf16x8 q[C::kSteps];
        {
            // a slot that is not there takes the block's first one's
            const int of = live ? slot : index * SharedPlan::kSlots;
            const int row = (int)((unsigned)of / (unsigned)a.group);
            const int head = h * a.group + of - row * a.group;
            const uint16_t* qp = static_cast<const uint16_t*>(a.q) +
                                 (int64_t)(lo + row) * a.q_ld + (int64_t)head * D + g * 8;
#pragma unroll
            for (int st = 0; st < C::kSteps; ++st) {
                const uint4 w = *reinterpret_cast<const uint4*>(qp + st * 16);
                q[st] = as_bf16x8(w.x, w.y, w.z, w.w);
            }
        }
        // waited for here, not among the loads of a tile
#pragma unroll
        for (int st = 0; st < C::kSteps; ++st) asm volatile("" : "+v"(q[st]));
        // The scale is taken as positive (products change their sign with it), so that
        // the largest product is the largest score and a masked -inf stays one; 0 as 1 of
        // products that are 0.
        const float signed_scale =
            a.scale * kLog2e * (F8 && c.k_scale != nullptr ? c.k_scale[h] : 1.0f);
        const float scale = signed_scale == 0.0f ? 1.0f : fabsf(signed_scale);
        const float sign = signed_scale == 0.0f ? 0.0f : signed_scale < 0.0f ? -1.0f : 1.0f;

        f32x16 acc[C::kDims];
#pragma unroll
        for (int i = 0; i < C::kDims; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][e] = 0.0f;
        // m (-inf: no score yet; else an integer), the m used, the product from which m is
        // raised, the lane's sum
        float m = -kInf, mu = 0.0f, far = -kInf, l = 0.0f;
        // The weights that are not yet multiplied with their values, as two bf16 terms (see
        // attend_kernel): a word two positions, 4 words an operand.
        uint32_t hi_w[8] = {}, rest_w[8] = {};
        auto value = [&](const char* values, int i) __attribute__((always_inline)) {
            // i: 32 dims i / 2, 16 positions i % 2
            const char* at = values + (i & 1) * 2 * C::kGroup + (i >> 2) * 1024;
            const s16x4 x0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4*)(at + v_at[0][(i >> 1) & 1]));
            const s16x4 x1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4*)(at + v_at[1][(i >> 1) & 1]));
            uint2 w0, w1;
            __builtin_memcpy(&w0, &x0, 8);
            __builtin_memcpy(&w1, &x1, 8);
            return as_bf16x8(w0.x, w0.y, w1.x, w1.y);
        };
        constexpr int kOperands = 2 * C::kDims, kAhead = 4;
        static_assert(kOperands == C::kSteps && kOperands >= kAhead, "");
        // the keys of a tile, operand A of every step
        bf16x8 k8[C::kSteps];
        auto key = [&](const char* keys, int st) __attribute__((always_inline)) {
            const uint4 w =
                *reinterpret_cast<const uint4*>(keys + k_at[st & 3] + (st >> 2) * 1024);
            k8[st] = as_bf16x8(w.x, w.y, w.z, w.w);
        };
        if constexpr (F8) {
            widen(sm.keys[0], 1);
            bring_all(sm.key_at[place(1)], nullptr, 1);
            bring_all(sm.value_at[place(0)], nullptr, 0);
        } else {
            asm volatile("s_waitcnt vmcnt(%0)" : : "n"(4 * C::kLoads) : "memory");
        }
        __syncthreads();
#pragma unroll
        for (int st = 0; st < C::kSteps; ++st) key(sm.keys[0], st);
        const char* next_k = sm.key_at[place(F8 ? 2 : 3)];
        const char* next_v = sm.value_at[place(F8 ? 1 : 2)];
        int in_keys = 1;  // of three: where the keys of tile t + 1 are
        // One turn: the scores of tile t, whose keys are in registers, then its weights
        // between the products of tile t - 1's with their values (BEHIND: there is one) and
        // the loads of the next tile's keys.  Behind the turn's only barrier the keys of
        // t + 1 and the values of t are in LDS, and the room of the keys of t and the
        // values of t - 2 is free.
        auto turn = [&](auto behind, int t) __attribute__((always_inline)) {
            constexpr bool kBehind = decltype(behind)::value;
            const int t0 = begin + t * C::kTile;
            f32x16 sc;
#pragma unroll
            for (int e = 0; e < 16; ++e) sc[e] = 0.0f;
#pragma unroll
            for (int st = 0; st < C::kSteps; ++st)
                sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k8[st], q[st], sc, 0, 0, 0);
            bf16x8 v8[kAhead];
            const char* values_behind = sm.values[(t + 3) & 3];
            if (kBehind)
#pragma unroll
                for (int i = 0; i < kAhead; ++i) v8[i] = value(values_behind, i);
            const bool masked =
                t0 + C::kTile > end || __builtin_amdgcn_readfirstlane(sm.holes) != 0;
            float p[16];  // position 8 (e / 4) + 4 g + e % 4
#pragma unroll
            for (int e = 0; e < 16; ++e) p[e] = sc[e];
            if (sign != 1.0f) {
#pragma unroll
                for (int e = 0; e < 16; ++e) p[e] *= sign;
            }
            if (masked) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t no = *reinterpret_cast<const uint32_t*>(
                        &sm.absent[(t * C::kTile + 8 * i + 4 * g) & (C::kPlaces - 1)]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if ((no >> (8 * e)) & 1) p[4 * i + e] = -kInf;
                }
            }
            float mx = p[0];
#pragma unroll
            for (int e = 1; e < 16; ++e) mx = fmaxf(mx, p[e]);
            // in the first tile, and hardly ever later
            if (__ballot(mx > far || (!F8 && l > C::kFull)) != 0) {
                const float top = fmaxf(mx, __shfl_xor(mx, 32));
                float to = fmaxf(m, ceilf(top * scale) + C::kHold);
                if (!F8 && fmaxf(l, __shfl_xor(l, 32)) > C::kFull) to += C::kRaise;
                if (to > m) {
                    // m = -inf: 0; else a power of two, as m is an integer
                    const float f = fast_exp2(m - to);
                    if (kBehind) {
#pragma unroll
                        for (int i = 0; i < C::kDims; ++i) acc[i] *= f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            hi_w[i] = pack_bf16(bf16_lo(hi_w[i]) * f, bf16_hi(hi_w[i]) * f);
                            rest_w[i] = pack_bf16(bf16_lo(rest_w[i]) * f, bf16_hi(rest_w[i]) * f);
                        }
                    }
                    l *= f;
                    m = mu = to;
                    far = (to - C::kHold + C::kSlack) / scale;
                }
            }
            const char* next_keys = sm.keys[in_keys];
            if constexpr (F8) {
                widen(sm.keys[in_keys], 1);
                widen(sm.values[t & 3], 0);
            } else {
                // all but the keys of t + 2 and the values of t + 1
                asm volatile("s_waitcnt vmcnt(%0)" : : "n"(2 * C::kLoads) : "memory");
            }
            __syncthreads();
            in_keys = in_keys == 2 ? 0 : in_keys + 1;
            char* into_keys = F8 ? nullptr : sm.keys[in_keys == 2 ? 0 : in_keys + 1];
            char* into_values = F8 ? nullptr : sm.values[(t + 2) & 3];
            if (kBehind && (t * C::kTile & (C::kPlaces / 2 - 1)) == 0)
                fetch_places(t0 + C::kPlaces / 2, C::kPlaces / 2);
            uint32_t new_hi[8], new_rest[8];
            constexpr float kOneUp = 1.0f + 0x1p-23f;
            // word i of the eight: a quarter of its work at a time
            auto weigh = [&](int i, int part) __attribute__((always_inline)) {
                float &x = p[2 * i], &y = p[2 * i + 1];
                if (part == 0) {
                    x = fast_exp2(fmaf(x, scale, -mu));
                    y = fast_exp2(fmaf(y, scale, -mu));
                } else if (part == 1) {
                    l += x;
                    new_hi[i] = __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x),
                                                      0x07060302u);
                } else if (part == 2) {
                    l += y;
                    x = fmaf(x, kOneUp, -bf16_hi(__float_as_uint(x)));
                } else {
                    y = fmaf(y, kOneUp, -bf16_hi(__float_as_uint(y)));
                    new_rest[i] = pack_bf16(x, y);
                }
            };
            if (kBehind) {
                // the words' 32 quarters spread over the 2 kOperands products
                constexpr int kEach = 16 / kOperands;
#pragma unroll
                for (int i = 0; i < kOperands; ++i) {
                    const uint32_t *w = hi_w + 4 * (i & 1), *u = rest_w + 4 * (i & 1);
                    f32x16& to = acc[i >> 1];
                    to = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        v8[i % kAhead], as_bf16x8(w[0], w[1], w[2], w[3]), to, 0, 0, 0);
#pragma unroll
                    for (int k = 2 * i * kEach; k < (2 * i + 1) * kEach; ++k)
                        weigh(k >> 2, k & 3);
                    __builtin_amdgcn_sched_barrier(0);
                    to = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        v8[i % kAhead], as_bf16x8(u[0], u[1], u[2], u[3]), to, 0, 0, 0);
#pragma unroll
                    for (int k = (2 * i + 1) * kEach; k < (2 * i + 2) * kEach; ++k)
                        weigh(k >> 2, k & 3);
                    if (i + kAhead < kOperands) v8[i % kAhead] = value(values_behind, i + kAhead);
                    key(next_keys, i);
                    // (all waves' loads at once would wait for each other)
                    if (i % 2 == 0) {
                        const int n = i / 2 % C::kLoads;
                        if (i / 2 < C::kLoads) bring(next_k, into_keys, 1, n);
                        else bring(next_v, into_values, 0, n);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            } else {
                bring_all(next_k, into_keys, 1);
                bring_all(next_v, into_values, 0);
#pragma unroll
                for (int k = 0; k < 32; ++k) weigh(k >> 2, k & 3);
#pragma unroll
                for (int st = 0; st < C::kSteps; ++st) key(next_keys, st);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                hi_w[i] = new_hi[i];
                rest_w[i] = new_rest[i];
                // made here, not where it is used
                asm volatile("" : "+v"(hi_w[i]), "+v"(rest_w[i]));
            }
            next_k = sm.key_at[place(t + (F8 ? 3 : 4))];
            next_v = sm.value_at[place(t + (F8 ? 2 : 3))];
        };
        turn(std::false_type{}, 0);
        int t = 1;
        if (t < n_tiles) {
            do {
                turn(std::true_type{}, t);
                ++t;
            } while (t < n_tiles);
        }
        // the last tile's weights
        if constexpr (!F8) {
            __builtin_amdgcn_s_waitcnt(0);  // its values, the last that were on their way
            __syncthreads();
        }
        {
            const char* values = sm.values[(n_tiles - 1) & 3];
            bf16x8 v8[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) v8[i] = value(values, i);
#pragma unroll
            for (int i = 0; i < kOperands; ++i) {
                const uint32_t *w = hi_w + 4 * (i & 1), *u = rest_w + 4 * (i & 1);
                f32x16& to = acc[i >> 1];
                to = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    v8[i % kAhead], as_bf16x8(w[0], w[1], w[2], w[3]), to, 0, 0, 0);
                to = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    v8[i % kAhead], as_bf16x8(u[0], u[1], u[2], u[3]), to, 0, 0, 0);
                if (i + kAhead < kOperands) v8[i % kAhead] = value(values, i + kAhead);
                __builtin_amdgcn_sched_barrier(0);
            }
        }

        l += __shfl_xor(l, 32);
        if (live) {
            const int64_t rec = (block_id + chunk) * SharedPlan::kSlots + wave * 32 + col;
            float* o = s.prefix_out + rec * D + 4 * g;
#pragma unroll
            for (int i = 0; i < C::kDims; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<f32x4*>(o + i * 32 + e * 8) =
                        f32x4{acc[i][4 * e], acc[i][4 * e + 1], acc[i][4 * e + 2],
                              acc[i][4 * e + 3]};
            if (g == 0) {
                s.prefix_ml[rec * 2] = m;
                s.prefix_ml[rec * 2 + 1] = l;
            }
        }
    }
    if (__ballot(bad) != 0 && lane == 0) raise_error(a.dev_error, SV_DEV_BAD_PAGE);
}

// Both kinds of workgroups: products keep those over the prefixes busy, loads of keys
// and values those over the requests' own positions, so that they share the CUs well,
// and small calls wait for one launch less.  One launch, and one after the other: 2 x 1
// row behind 512 positions 9.5 and 16.7 us, 48 x 1 .. 8 rows behind 2000 (8 bits) 25 and
// 36, 256 x 1 .. 8 rows (32 heads over 8, dim 128) behind 8192, up to 500 of their own,
// 274 and 311: 115 GFLOP over the prefix (173 with the weights' second terms, 630
// TFLOP/s) beside 290 MB read, at a clock that falls below 2 GHz under it.
template <int D, bool F8, int MT, bool PG16>
__global__ __launch_bounds__(256, (Prefix<D, F8>::kOccupancy)) void shared_kernel(SharedArgs s) {
    using Own = Attend<D, F8, MT, PG16>;
    static_assert(Own::kOccupancy >= Prefix<D, F8>::kOccupancy, "registers for both");
    __shared__ union {
        typename Prefix<D, F8>::Smem prefix;
        typename Own::Smem own;
    } sm;
    if ((int)blockIdx.x < s.chunks)
        prefix<D, F8>(s, blockIdx.x, sm.prefix);
    else
        attend_own<D, F8, MT, PG16>(s.own, blockIdx.x - s.chunks, gridDim.x - s.chunks, sm.own);
}

// --------------------------------------------------------------------- join

// Merges the parts of a row's heads, those over the prefix first, in a fixed order.  W
// waves take H neighbouring heads: lanes over the dims, wave w the parts w, w + W, ...; the
// waves' sums meet in LDS.  Bound by the latency of its loads, first of those that lead to
// the parts, then of the parts themselves: hipcc puts a part's load behind the test that
// ends the sum, so that of the first (or only) head one is on its way at a time, of the
// second four (256 x 1 .. 8 rows, 32 heads of 128: 37 us for 62 MB of parts).
template <int D, bool F8, int W, int H>
__global__ __launch_bounds__(256) void shared_join_kernel(SharedArgs s) {
    constexpr int E = D / kWave;
    constexpr int kMost = 128;  // parts
    __shared__ float factors[4][H][kMost];
    __shared__ float sums[W == 1 ? 1 : 4][D];
    const AttendArgs& a = s.own;
    const sv_cache& c = a.cache;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wave % W;
    const int runs = (a.n_heads + H - 1) / H;
    const int per = (a.k_max + 1) * runs;
    const int64_t id = (int64_t)blockIdx.x * (4 / W) + wave / W;
    if (id >= (int64_t)a.n_req * per) return;
    const int r = (int)(id / per), rest = (int)id - r * per;
    const int row = rest / runs, head0 = (rest - row * runs) * H;
    const int first = s.first[r];
    const int lo = a.cu_rows[r], hi = a.cu_rows[r + 1], rows = hi - lo, ctx = a.ctx_len[r];
    if (first < 0 || lo < 0 || hi < lo || rows > a.k_max + 1 || hi > a.q_rows || row >= rows ||
        ctx < first || (int64_t)ctx + rows > (int64_t)a.max_pages * c.page_size)
        return;
    // the parts as the launch before made them
    int n1[H], n[H];
    int64_t rec1[H];  // parts are kSlots records apart
    const int len = ctx + rows - (first & ~15), plen = part_len(len, a.parts, a.part_min);
    const int n2 = (len + plen - 1) / plen;
#pragma unroll
    for (int i = 0; i < H; ++i) n1[i] = 0, rec1[i] = 0;
    if (first > 0) {
        const SharedRequest at = s.request[r];
        const int head_blocks = s.group[s.n_groups].block, block0 = s.group[at.group].block;
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const int head = min(head0 + i, a.n_heads - 1), h = head / a.group;
            const int slot = (at.row + row) * a.group + head - h * a.group;
            const int64_t block_id =
                (int64_t)h * head_blocks + block0 + slot / SharedPlan::kSlots;
            const SharedSpan span = s.span[block_id];
            n1[i] = span.last - span.first + 1;
            rec1[i] = (block_id + span.first) * SharedPlan::kSlots + slot % SharedPlan::kSlots;
        }
    }
    int most = 0;
    float m[H], l[H], o[H][E];
    int64_t rec2[H];
#pragma unroll
    for (int i = 0; i < H; ++i) {
        const int head = min(head0 + i, a.n_heads - 1);
        n[i] = n1[i] + n2;  // at most kMost
        most = max(most, n[i]);
        // attend's records: request, head, row
        rec2[i] = (((int64_t)r * a.n_heads + head) * (a.k_max + 1) + row) * a.parts;
    }
    // the largest maximum and the parts' factors, two a lane
    float mm[H][2], ll[H][2];
#pragma unroll
    for (int i = 0; i < H; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            mm[i][j] = -kInf;
            ll[i][j] = 0.0f;
            const int p = lane + 64 * j;
            if (p >= n[i]) continue;
            const float* ml = p < n1[i] ? s.prefix_ml + (rec1[i] + p * SharedPlan::kSlots) * 2
                                        : a.part_ml + (rec2[i] + p - n1[i]) * 2;
            mm[i][j] = ml[0];
            ll[i][j] = ml[1];
        }
#pragma unroll
    for (int i = 0; i < H; ++i) {
        m[i] = wave_max(fmaxf(mm[i][0], mm[i][1]));
        float f[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            f[j] = mm[i][j] == m[i] ? 1.0f : fast_exp2(mm[i][j] - m[i]);
            ll[i][j] = lane + 64 * j < n[i] ? f[j] * ll[i][j] : 0.0f;
        }
        l[i] = wave_sum(ll[i][0] + ll[i][1]);
        // over the whole sum before the outputs are added up: they are then shares of the
        // mean, and stay in range
        const float inv = l[i] == 0.0f ? 0.0f : 1.0f / l[i];
        factors[wave][i][lane] = f[0] * inv;
        factors[wave][i][lane + 64] = f[1] * inv;
#pragma unroll
        for (int e = 0; e < E; ++e) o[i][e] = 0.0f;
    }
    __builtin_amdgcn_wave_barrier();
    for (int p0 = w; p0 < most; p0 += 4 * W) {
        float x[H][4][E];
#pragma unroll
        for (int i = 0; i < H; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int p = min(p0 + j * W, n[i] - 1);
                const float* from =
                    (p < n1[i] ? s.prefix_out + (rec1[i] + p * SharedPlan::kSlots) * D
                               : a.part_out + (rec2[i] + p - n1[i]) * D) +
                    lane * E;
#pragma unroll
                for (int e = 0; e < E; ++e) x[i][j][e] = from[e];
            }
#pragma unroll
        for (int i = 0; i < H; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (p0 + j * W >= n[i]) break;
                const float f = factors[wave][i][p0 + j * W];
#pragma unroll
                for (int e = 0; e < E; ++e) o[i][e] += f * x[i][j][e];
            }
    }
    if (W > 1) {
        static_assert(W == 1 || H == 1, "");
#pragma unroll
        for (int e = 0; e < E; ++e) sums[wave][lane * E + e] = o[0][e];
        __syncthreads();
        if (w != 0) return;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int i = lane * E + e;
            o[0][e] = (sums[0][i] + sums[1][i]) + (sums[2][i] + sums[3][i]);
        }
    }
#pragma unroll
    for (int i = 0; i < H; ++i) {
        const int head = head0 + i;
        if (head >= a.n_heads) break;
        const float vscale = F8 && c.v_scale != nullptr ? c.v_scale[head / a.group] : 1.0f;
        uint16_t* out = static_cast<uint16_t*>(a.out) + (int64_t)(lo + row) * a.out_ld +
                        (int64_t)head * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e)
            out[e] = (uint16_t)pack_bf16(l[i] == 0.0f ? 0.0f : o[i][e] * vscale, 0.0f);
        if (a.out_lse != nullptr && lane == 0) {
            // the sum's exponent first: both terms are then of the result's size
            int e;
            const float f = frexpf(l[i], &e);
            a.out_lse[(int64_t)(lo + row) * a.n_heads + head] =
                l[i] == 0.0f ? -kInf : ((m[i] + (float)e) + log2f(f)) * kLn2;
        }
    }
}

template <int D, bool F8>
void run_shared_join(const SharedArgs& s, hipStream_t stream) {
    const int64_t rows = (int64_t)s.own.n_req * (s.own.k_max + 1);
    // Few rows: a workgroup a head, so that four parts are read at once (16 rows of 32 heads,
    // 64 parts, 14.9 -> 6.9 us; 384 of 16 heads, a few parts, 8.9 -> 14.2).  Many: two heads
    // a wave (one, two, four: whole calls of 256 x 1 .. 8 rows 316, 313, 310 us, of 48 x
    // 1 .. 8 rows 41.1, 41.7, 44.2).
    if (rows * s.own.n_heads <= 2048) {
        shared_join_kernel<D, F8, 4, 1><<<(unsigned)(rows * s.own.n_heads), 256, 0, stream>>>(s);
    } else {
        const int64_t runs = rows * ((s.own.n_heads + 1) / 2);
        shared_join_kernel<D, F8, 1, 2><<<(unsigned)((runs + 3) / 4), 256, 0, stream>>>(s);
    }
}

template <int D, bool F8, int MT>
void run_both(const SharedArgs& s, hipStream_t stream) {
    const AttendArgs& a = s.own;
    const unsigned grid = (unsigned)(s.chunks + (int64_t)a.cache.n_kv_heads * a.n_req *
                                                    a.slot_blocks * a.parts);
    if (a.cache.page_size % 16 == 0 && 16 * a.cache.token_stride <= (int64_t)1 << 28)
        shared_kernel<D, F8, MT, true><<<grid, 256, 0, stream>>>(s);
    else
        shared_kernel<D, F8, MT, false><<<grid, 256, 0, stream>>>(s);
}

template <int D, bool F8>
hipError_t run_shared(const SharedArgs& s, hipStream_t stream) {
    const AttendArgs& a = s.own;
    if (a.n_req <= 256) layout_kernel<256, true><<<1, 256, 0, stream>>>(s);
    else if (a.n_req <= 1024) layout_kernel<1024, true><<<1, 1024, 0, stream>>>(s);
    else layout_kernel<1024, false><<<1, 1024, 0, stream>>>(s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // the plan takes slot_tiles * D <= 256
    if (a.slot_tiles == 1) run_both<D, F8, 1>(s, stream);
    else if constexpr (D == 256) return hipErrorInvalidValue;
    else if (a.slot_tiles == 2) run_both<D, F8, 2>(s, stream);
    else if constexpr (D == 128) return hipErrorInvalidValue;
    else run_both<D, F8, 4>(s, stream);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    run_shared_join<D, F8>(s, stream);
    return hipGetLastError();
}

template <int D>
hipError_t run_shared_d(const SharedArgs& s, hipStream_t stream) {
    return s.own.cache.dtype == SV_E4M3 ? run_shared<D, true>(s, stream)
                                        : run_shared<D, false>(s, stream);
}

}  // namespace

hipError_t launch_cache_attend_shared(const SharedArgs& a, hipStream_t stream) {
    switch (a.own.cache.head_dim) {
        case 64: return run_shared_d<64>(a, stream);
        case 128: return run_shared_d<128>(a, stream);
        default: return run_shared_d<256>(a, stream);
    }
}

}  // namespace sv
