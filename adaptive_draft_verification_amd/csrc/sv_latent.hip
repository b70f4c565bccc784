// The paged cache of latent vectors (gfx950, wave64): sv_latent_append writes a
// step's vectors behind each request's context, sv_latent_attend lets the packed
// rows of every head attend to them.
#include "sv_attend.h"
#include "sv_device.h"
#include "sv_latent.h"
#include "sv_launch.h"

namespace sv {
namespace {

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
// i % H): all of them read the same vectors.  A workgroup of four waves takes 64
// slots over one part of the cached positions, 32 of them at a time, which lie in
// LDS as bf16.  A pair of waves takes 32 slots.  Each of the two takes the scores
// of 16 positions over all dims and half of the output's dims over all 32 positions,
// so that the accumulators are R / 4 registers a lane beside R / 4 + 16 of queries;
// the weights of the other 16 positions come from the other wave through LDS.
// At 512 dims a few values that only the ends of a part need do not fit beside them and go
// to scratch (16 bytes a lane; 56 with 8-bit tiles, which pass registers): none is read
// back within a turn.
// Operands:
//   S^T = K Q^T, v_mfma_f32_16x16x32_bf16: A holds 16 positions (lane % 16) by 32 dims
//   (8 for each g = lane / 16), B 16 slots by the same dims, so a lane ends with the
//   scores of ONE slot (lane % 16) at positions 4 g .. 4 g + 3;
//   O^T = C^T P^T, v_mfma_f32_32x32x16_bf16: B's lane holds 8 positions, 8 (lane / 32)
//   .. of either wave's 16, of slot lane % 32, which one exchange of 16 lanes makes of
//   both slots' weights; A needs the same positions of one dim a lane: two transposing
//   LDS reads of 4 positions by 16 dims for each 16 lanes.
// A KB read from LDS feeds 32 clocks of products with keys and 64 with values: 95
// of the 128 bytes a clock that LDS gives at full rate.  The weights of a tile are
// taken between the products of the tile before with its values: one wave a SIMD
// has the registers, so nothing else would fill that time.
// In LDS 8 positions by 8 chunks of 16 bytes are a KB, the chunk c of position x at
// (c ^ swizzle(x)) of its 128 bytes.  LDS has 64 banks of 4 bytes: the chunk c of 16
// neighbouring positions, and the chunks c and c ^ 1 of 8, lie in different ones.
// A load brings one such KB, 8 lanes a position.
// Bound by the products and what stands between them: a turn of 32 positions takes a wave
// some 3500 clocks, 1600 of them products (scores 1080 with their keys' way from LDS,
// values 1250, the next tile's addresses, maxima, exchange and barriers the rest).  128
// x 1 .. 8 rows of 128 heads on up to 4096 positions 718 us, 2 x 8 rows on 100,000 620 us:
// 720 TFLOP/s, 1060 with the weights' second terms, where a large product of this card's
// library reaches 1230.

__device__ __forceinline__ int swizzle(int pos) { return (pos & 6) | ((pos >> 3) & 1); }

// What a position without a page is loaded from.
__device__ const uint4 kZeros[(512 + SV_LATENT_ROPE) / 8] = {};

template <int R, bool F8>
struct Latent {
    static constexpr int kTile = 32, kSlots = 64;
    static constexpr int kDim = R + SV_LATENT_ROPE, kChunks = kDim / 8;
    static constexpr int kGroup = kDim * 2 * 8;    // bytes of 8 positions
    static constexpr int kTileBytes = 4 * kGroup;  // a group a wave
    static constexpr int kLoads = kChunks / 8;     // of a group
    static constexpr int kSteps = kDim / 32;       // products of a score
    static constexpr int kEarly = kSteps / 4;      // loads issued between them
    static constexpr int kDims = R / 64;           // 32-dim tiles of a wave's output
    static constexpr int kEsize = F8 ? 1 : 2;
    static constexpr int kPlaces = 1024;           // positions whose places are in LDS
    // Weights are 2^(score - m), m kHold above the maximum of the slot's first tile.
    // They are 2^-32 at most while no score passes that maximum by 2^kSlack, so that
    // sums over 2^31 positions stay below 1 and sums of weighted values in fp32's
    // range, however large the values are.  Where one does, which is rare, the
    // workgroup starts again from the true maxima.
    static constexpr float kHold = 64.0f, kSlack = 32.0f;
};

template <int R, bool F8>
__global__ __launch_bounds__(256, 1) void latent_kernel(LatentAttendArgs a) {
    using C = Latent<R, F8>;
    __shared__ __attribute__((aligned(16))) char tiles[3][C::kTileBytes];
    __shared__ uint4 weights[2][4][2][kWave];  // of even and odd tiles: a wave's, for the other
    __shared__ float tops[4][32];              // maxima of a wave's slots
    // of position begin + i at i % kPlaces: where it is, and whether there is none
    __shared__ const char* places[C::kPlaces];
    __shared__ __attribute__((aligned(4))) uint8_t absent[C::kPlaces];
    // a byte a position of the tile: it is not finite
    __shared__ __attribute__((aligned(4))) uint8_t tainted[3][C::kTile];
    __shared__ int holes;     // a position before the end is none
    __shared__ int risen[2];  // a score passed its slot's m by too much, in an even or odd tile
    const sv_latent_cache& c = a.cache;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int pair = wave >> 1, half = wave & 1;
    // grid: slot blocks fastest, then requests and parts
    int id = spread(blockIdx.x, gridDim.x, a.slot_blocks);
    const int mb = id % a.slot_blocks;
    id /= a.slot_blocks;
    int r = id % a.n_req;
    const int part = id / a.n_req;
    if (a.longest_first) r = longest(r, a.ctx_len, a.n_req, reinterpret_cast<int*>(tiles));

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
    const int slots = rows * a.n_heads - mb * C::kSlots;  // slots of this block
    if (slots <= 0) return;
    const int len = ctx + rows;
    const int plen = latent_part_len(len, a.parts, a.part_min);
    const int begin = part * plen, end = min(len, begin + plen);
    if (begin >= len) return;
    const bool whole = plen >= len;  // the request's only part

    // ---- the vectors' way into LDS: wave w brings positions 8 w .. 8 w + 7 of a tile
    const char* kv = static_cast<const char*>(c.kv);
    const int32_t* table = a.page_table + (int64_t)r * a.max_pages;
    const int mine = wave * 8 + (lane >> 3);
    const int chunk_of = ((lane & 7) ^ swizzle(mine)) * 8 * C::kEsize;
    // The places of `n` positions from `from` on, into LDS: kPlaces at first, then half
    // as many at a time (a wait for a page id in registers would be a wait for the tile
    // that is on its way).  None: after the end, or on a page that is not there.
    auto fetch_places = [&](int from, int n) __attribute__((always_inline)) {
        for (int i = threadIdx.x; i < n; i += 256) {
            const int64_t t = (int64_t)from + i;
            const char* at = reinterpret_cast<const char*>(kZeros);
            bool none = true;
            if (t < end) {
                const int in = a.page_shift >= 0
                                   ? (int)t >> a.page_shift
                                   : (int)((unsigned)t / (unsigned)c.page_size);
                const int page = table[in];
                if (page >= 0 && page < c.n_pages) {
                    at = kv + ((int64_t)page * c.page_stride +
                               (int64_t)((int)t - in * c.page_size) * c.token_stride) *
                                  C::kEsize;
                    none = false;
                } else {
                    holes = 1;
                }
            }
            places[(int)(t - begin) & (C::kPlaces - 1)] = at;
            absent[(int)(t - begin) & (C::kPlaces - 1)] = none;
        }
    };
    auto look_up = [&](int t0) { return places[(t0 + mine - begin) & (C::kPlaces - 1)]; };
    uint2 raw[F8 ? C::kLoads : 1];
    const char* from;
    uint32_t to_lds;
    // the loads of a tile are made ready, and then issued one by one
    auto prepare = [&](int buf, const char* place) __attribute__((always_inline)) {
        from = place + chunk_of;
        to_lds = __builtin_amdgcn_readfirstlane(lds_address(tiles[buf] + wave * C::kGroup));
    };
    auto issue = [&](int i) __attribute__((always_inline)) {
        if constexpr (F8) raw[i] = load_global8(from + i * 64);
        else load_to_lds<128>(from, to_lds + i * 1024, i);
    };
    // the first tile's
    auto start = [&]() __attribute__((always_inline)) {
        fetch_places(begin, C::kPlaces);
        __syncthreads();
        prepare(0, look_up(begin));
#pragma unroll
        for (int i = 0; i < C::kLoads; ++i) issue(i);
        return look_up(begin + C::kTile);
    };
    // an 8-bit tile goes into LDS as bf16 when it has arrived
    auto settle = [&](int buf) __attribute__((always_inline)) {
        if constexpr (F8) {
#pragma unroll
            for (int i = 0; i < C::kLoads; ++i)
                *reinterpret_cast<uint4*>(tiles[buf] + wave * C::kGroup + i * 1024 + lane * 16) =
                    make_uint4(e4m3_pair<false>(raw[i].x), e4m3_pair<true>(raw[i].x),
                               e4m3_pair<false>(raw[i].y), e4m3_pair<true>(raw[i].y));
        }
        __builtin_amdgcn_s_waitcnt(0);
    };

    // the order of requests was read from where the tiles go
    if (threadIdx.x == 0) risen[0] = risen[1] = holes = 0;
    __syncthreads();
    const char* place = start();

    // ---- queries of the pair's slots, operand B of every step
    int q_row[2], head[2], last[2];  // last: the position a slot sees last
    bool live[2];
    const uint16_t* q_at[2];
#pragma unroll
    for (int sh = 0; sh < 2; ++sh) {
        const int i = pair * 32 + sh * 16 + col, slot = mb * C::kSlots + i;
        live[sh] = i < slots;
        q_row[sh] = (int)((unsigned)slot / (unsigned)a.n_heads);
        head[sh] = slot - q_row[sh] * a.n_heads;
        last[sh] = live[sh] ? ctx + q_row[sh] : -1;
        // a slot that is not there takes the first one's: it sees nothing
        q_at[sh] = static_cast<const uint16_t*>(a.q) +
                   (int64_t)(live[sh] ? lo + q_row[sh] : lo) * a.q_ld +
                   (int64_t)(live[sh] ? head[sh] : 0) * C::kDim + g * 8;
    }
    bf16x8 q[C::kSteps][2];
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int st = 0; st < C::kSteps; ++st)
#pragma unroll
        for (int sh = 0; sh < 2; ++sh) {
            const uint4 w = *reinterpret_cast<const uint4*>(q_at[sh] + st * 32);
            q[st][sh] = as_bf16x8(w.x, w.y, w.z, w.w);
        }
    __builtin_amdgcn_sched_barrier(0);
    // Waited for here, not among the loads of a tile.  512 registers a lane are 256 for
    // any use and 256 for products alone: most of the queries go among the latter.
#pragma unroll
    for (int st = 0; st < C::kSteps; ++st)
        if (st < 4) asm volatile("" : "+v"(q[st][0]), "+v"(q[st][1]));
        else asm volatile("" : "+a"(q[st][0]), "+a"(q[st][1]));

    // The scale is taken as positive (products change their sign with it), so that the
    // largest product is the largest score and a masked -inf stays one; 0 as 1 of
    // products that are 0.
    const float kv_scale = F8 && c.scale != nullptr ? *c.scale : 1.0f;
    const float signed_scale = a.scale * kLog2e * kv_scale;
    const float scale = signed_scale == 0.0f ? 1.0f : fabsf(signed_scale);
    const float sign = signed_scale == 0.0f ? 0.0f : signed_scale < 0.0f ? -1.0f : 1.0f;

    f32x16 acc[C::kDims];
    float m[2], mu[2];  // m (-inf: no score in the first tile), the m used
    float far[2];       // the product whose score is kSlack above the first ones
    float l[2];         // sum

    // where a lane reads keys: chunks 4 st + g of its position, st = 0, 1 of 128 bytes
    int k_at[2], v_own[2], v_other[2];
    {
        const int pos = half * 16 + col, at = (pos >> 3) * C::kGroup + (pos & 7) * 128;
#pragma unroll
        for (int j = 0; j < 2; ++j) k_at[j] = at + ((4 * j + g) ^ swizzle(pos)) * 16;
    }
    // and values: 4 positions by 16 dims for 16 lanes, the first four of 8 and even 32
    // dims or the second and odd ones, then the others; of the wave's half of the dims, of
    // its own positions and of the other wave's
    {
        const int pos = 8 * (lane >> 5) + ((lane & 15) >> 2);
        const int at = (pos >> 3) * C::kGroup + (pos & 7) * 128 + (lane & 1) * 8 +
                       half * (R / 128) * 1024;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int ch = 4 * j + 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
            const int x = at + (ch ^ swizzle(pos)) * 16;
            v_own[j] = x + half * 2 * C::kGroup;
            v_other[j] = x + (half ^ 1) * 2 * C::kGroup;
        }
    }

    // The tile at t0 has arrived: makes the next one's loads ready (after the end they
    // bring zeros), and cleans this one where it holds the step's own rows.
    auto enter = [&](int t0, int buf) __attribute__((always_inline)) {
        prepare(buf == 2 ? 0 : buf + 1, place);
        place = look_up(t0 + 2 * C::kTile);
        if (t0 > begin && ((t0 - begin) & (C::kPlaces / 2 - 1)) == 0)
            fetch_places(t0 + C::kPlaces / 2, C::kPlaces / 2);
        if (t0 + C::kTile > ctx) {
            // These rows do not all see each other: a vector that is not finite may
            // touch only those that see it.  It is zeroed, and its score is NaN.
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
                if (lane == 0) tainted[buf][wave * 8 + i] = 0;
                if (t0 + wave * 8 + i <= ctx) continue;
                uint4* at = reinterpret_cast<uint4*>(tiles[buf] + wave * C::kGroup + i * 128 +
                                                     (lane >> 3) * 1024 + (lane & 7) * 16);
                bool nf = false;
                for (int ch = 0; ch < C::kChunks; ch += kWave) {
                    if (ch + lane >= C::kChunks) break;
                    const uint4 w = at[ch * 8];
                    nf |= bf16_pair_nonfinite(w.x) || bf16_pair_nonfinite(w.y) ||
                          bf16_pair_nonfinite(w.z) || bf16_pair_nonfinite(w.w);
                }
                if (__ballot(nf) == 0) continue;
                if (lane == 0) tainted[buf][wave * 8 + i] = 1;
                for (int ch = 0; ch < C::kChunks; ch += kWave)
                    if (ch + lane < C::kChunks) at[ch * 8] = make_uint4(0, 0, 0, 0);
            }
            __syncthreads();
        }
    };
    // The products of the lane's four positions and two slots.  Between two matrix
    // instructions there is time for three others: the keys' reads, kAhead steps before
    // their products, and the first of the next tile's loads.
    auto score = [&](int t0, int buf, float (&p)[2][4], auto behind)
                     __attribute__((always_inline)) {
        const char* tile = tiles[buf];
        const int any_hole = holes;
        auto key = [&](int st) __attribute__((always_inline)) {
            const uint4 w = *reinterpret_cast<const uint4*>(tile + k_at[st & 1] + (st >> 1) * 1024);
            return as_bf16x8(w.x, w.y, w.z, w.w);
        };
        // two sums a slot: a product waits for the one before it on the same sum
        constexpr int kAhead = 5;
        f32x4 s[2][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i >> 1][i & 1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        bf16x8 k8[kAhead];
#pragma unroll
        for (int st = 0; st < kAhead; ++st) k8[st] = key(st);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int st = 0; st < C::kSteps; ++st) {
            s[0][st & 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k8[st % kAhead], q[st][0],
                                                                   s[0][st & 1], 0, 0, 0);
            if (st % 4 == 1 && st / 4 < C::kEarly) issue(st / 4);
            __builtin_amdgcn_sched_barrier(0);
            s[1][st & 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k8[st % kAhead], q[st][1],
                                                                   s[1][st & 1], 0, 0, 0);
            if (st + kAhead < C::kSteps) k8[st % kAhead] = key(st + kAhead);
            __builtin_amdgcn_sched_barrier(0);
        }
        behind();  // while the last products are on their way
#pragma unroll
        for (int sh = 0; sh < 2; ++sh)
#pragma unroll
            for (int e = 0; e < 4; ++e) p[sh][e] = (s[sh][0][e] + s[sh][1][e]) * sign;
        const bool edge = t0 + C::kTile > ctx;
        if (edge || __builtin_amdgcn_readfirstlane(any_hole) != 0) {
            const int first = half * 16 + 4 * g;
            const uint32_t no = *reinterpret_cast<const uint32_t*>(&absent[(t0 - begin + first) & (C::kPlaces - 1)]);
            const uint32_t nan =
                edge ? *reinterpret_cast<const uint32_t*>(&tainted[buf][first]) : 0;
#pragma unroll
            for (int sh = 0; sh < 2; ++sh) {
                const int sees = last[sh] - (t0 + first);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if ((nan >> (8 * e)) & 1) p[sh][e] = __builtin_nanf("");
                    if (((no >> (8 * e)) & 1) || e > sees) p[sh][e] = -kInf;
                }
            }
        }
    };
    // Over the lanes of a slot.
    auto top_of = [&](float x) {
        x = fmaxf(x, __shfl_xor(x, 16));
        return fmaxf(x, __shfl_xor(x, 32));
    };
    // The pair's maximum of both slots, from each lane's own.
    auto exchange = [&](float (&x)[2]) __attribute__((always_inline)) {
#pragma unroll
        for (int sh = 0; sh < 2; ++sh) {
            x[sh] = top_of(x[sh]);
            if (g == 0) tops[wave][sh * 16 + col] = x[sh];
        }
        __syncthreads();
#pragma unroll
        for (int sh = 0; sh < 2; ++sh) x[sh] = fmaxf(x[sh], tops[wave ^ 1][sh * 16 + col]);
    };

    auto refer = [&](const float (&top)[2]) {
#pragma unroll
        for (int sh = 0; sh < 2; ++sh) {
            m[sh] = top[sh] * scale + C::kHold;
            mu[sh] = m[sh] == -kInf ? 0.0f : m[sh];
            // (-inf also where a scale near zero makes the distance infinite)
            far[sh] = top[sh] == -kInf ? -kInf : top[sh] + C::kSlack / scale;
        }
    };
    // Weights go into the product as two bf16 terms, the upper half of the fp32 weight
    // and the rest, off by at most 2^-15 of each: one term's 2^-8 would show in the
    // result beside its own rounding.  Both are positive where the weight is (the rest
    // of 1 + 2^-23 times it is taken): an infinite value times 0 or a negative rest
    // would make NaN.
    auto weigh = [&](float& x, int sh) __attribute__((always_inline)) {
        x = fast_exp2(fmaf(x, scale, -mu[sh]));
        l[sh] += x;
        asm volatile("" : "+v"(x));  // here, not where it is used
    };
    auto split = [&](const float (&p)[4]) __attribute__((always_inline)) {
        constexpr float kOneUp = 1.0f + 0x1p-23f;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float x = p[2 * i], y = p[2 * i + 1];
            const uint32_t xb = __float_as_uint(x), yb = __float_as_uint(y);
            w[i] = __builtin_amdgcn_perm(yb, xb, 0x07060302u);
            w[2 + i] = pack_bf16(fmaf(x, kOneUp, -bf16_hi(xb)), fmaf(y, kOneUp, -bf16_hi(yb)));
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    };
    // Words of both slots' splits as operands: the lane's slot is lane % 32 then, its
    // positions 8 (lane / 32) .. of 16.
    struct Weights {
        uint4 hi, rest;
    };
    auto operands = [&](const uint4& x, const uint4& y) __attribute__((always_inline)) {
        const auto h0 = __builtin_amdgcn_permlane16_swap(x.x, y.x, false, false);
        const auto h1 = __builtin_amdgcn_permlane16_swap(x.y, y.y, false, false);
        const auto r0 = __builtin_amdgcn_permlane16_swap(x.z, y.z, false, false);
        const auto r1 = __builtin_amdgcn_permlane16_swap(x.w, y.w, false, false);
        return Weights{make_uint4(h0[0], h1[0], h0[1], h1[1]),
                       make_uint4(r0[0], r1[0], r0[1], r1[1])};
    };

    // a second time from the true maxima, if a score rose too far above the first ones
    for (bool again = false;; again = true) {
#pragma unroll
        for (int i = 0; i < C::kDims; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][e] = 0.0f;
        l[0] = l[1] = 0.0f;
        if (again) place = start();
        Weights own;  // of the tile before
        {
            settle(0);
            __syncthreads();
            enter(begin, 0);
            float p[2][4];
            score(begin, 0, p, [] {});
#pragma unroll
            for (int i = C::kEarly; i < C::kLoads; ++i) issue(i);
            if (!again) {
                float mx[2];
#pragma unroll
                for (int sh = 0; sh < 2; ++sh)
                    mx[sh] = fmaxf(fmaxf(p[sh][0], p[sh][1]), fmaxf(p[sh][2], p[sh][3]));
                exchange(mx);
                refer(mx);
            }
#pragma unroll
            for (int sh = 0; sh < 2; ++sh)
#pragma unroll
                for (int e = 0; e < 4; ++e) weigh(p[sh][e], sh);
            own = operands(split(p[0]), split(p[1]));
            weights[0][wave][0][lane] = own.hi;
            weights[0][wave][1][lane] = own.rest;
        }
        // a turn takes the scores of its tile (there is none in the last turn) and the
        // values of the one before
        bool rose = false, more = true;
        int buf = 1, odd = 1;
        for (int t0 = begin + C::kTile; more; t0 += C::kTile) {
            settle(buf);
            __syncthreads();
            // of the tile before: no wave is a tile further before this one has read it
            const int rose_before = risen[odd ^ 1];
            const Weights other{weights[odd ^ 1][wave ^ 1][0][lane],
                                weights[odd ^ 1][wave ^ 1][1][lane]};
            more = t0 < end;
            const char* tile = tiles[buf == 0 ? 2 : buf - 1];
            // value operand i: dims 32 (i / 2) .., the wave's own 16 positions or the other's
            auto value = [&](int i) __attribute__((always_inline)) {
                const char* at = tile + (i >> 2) * 1024;
                const int j = (i >> 1) & 1;
                const s16x4 x0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3)))
                     s16x4*)(at + ((i & 1) == 0 ? v_own[j] : v_other[j])));
                const s16x4 x1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3)))
                     s16x4*)(at + 512 + ((i & 1) == 0 ? v_own[j ^ 1] : v_other[j ^ 1])));
                uint2 w0, w1;
                __builtin_memcpy(&w0, &x0, 8);
                __builtin_memcpy(&w1, &x1, 8);
                return as_bf16x8(w0.x, w0.y, w1.x, w1.y);
            };
            constexpr int kAhead = 4;
            bf16x8 v8[kAhead];
            auto first_values = [&]() __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) v8[i] = value(i);
                __builtin_amdgcn_sched_barrier(0);
            };
            float p[2][4];
            if (more) {
                enter(t0, buf);
                score(t0, buf, p, first_values);
                bool above = false;
#pragma unroll
                for (int sh = 0; sh < 2; ++sh)
                    above |= fmaxf(fmaxf(p[sh][0], p[sh][1]), fmaxf(p[sh][2], p[sh][3])) > far[sh];
                if (__ballot(above) != 0) risen[odd] = 1;
            } else {
                first_values();
#pragma unroll
                for (int e = 0; e < 8; ++e) p[e >> 2][e & 3] = -kInf;
            }
            rose = !again && __builtin_amdgcn_readfirstlane(rose_before) != 0;
            more = more && !rose;
            uint4 words[2];
            // Between the products the values' reads, kAhead operands ahead, this turn's
            // weights and the rest of the next tile's loads (in the last turn weights of 0,
            // and loads to where nothing is read any more).
            constexpr int kProducts = 4 * C::kDims;
#pragma unroll
            for (int k = 0; k < kProducts; ++k) {
                const int i = k >> 1;
                const Weights& of = (i & 1) == 0 ? own : other;
                const uint4& w = (k & 1) == 0 ? of.hi : of.rest;
                acc[i >> 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    v8[i % kAhead], as_bf16x8(w.x, w.y, w.z, w.w), acc[i >> 1], 0, 0, 0);
                constexpr int kEvery = kProducts / 16;  // 8 weights in half of the products
                if (k % kEvery == 0 && k / kEvery < 8)
                    weigh(p[k / kEvery >> 2][k / kEvery & 3], k / kEvery >> 2);
                if (k == kProducts / 2) words[0] = split(p[0]);
                if (k == kProducts / 2 + 2) words[1] = split(p[1]);
                if (k % 4 == 1 && C::kEarly + k / 4 < C::kLoads) issue(C::kEarly + k / 4);
                if ((k & 1) == 1 && i + kAhead < 2 * C::kDims) v8[i % kAhead] = value(i + kAhead);
                __builtin_amdgcn_sched_barrier(0);
            }
            own = operands(words[0], words[1]);
            weights[odd][wave][0][lane] = own.hi;
            weights[odd][wave][1][lane] = own.rest;
            buf = buf == 2 ? 0 : buf + 1;
            odd ^= 1;
        }
        __builtin_amdgcn_s_waitcnt(0);  // nothing is on its way to LDS
        if (!rose) break;
        __syncthreads();  // every wave has left the tiles
        place = start();
        float mx[2] = {-kInf, -kInf};
        buf = 0;
        for (int t0 = begin; t0 < end; t0 += C::kTile, buf = buf == 2 ? 0 : buf + 1) {
            settle(buf);
            __syncthreads();
            enter(t0, buf);
            float p[2][4];
            score(t0, buf, p, [] {});
#pragma unroll
            for (int i = C::kEarly; i < C::kLoads; ++i) issue(i);
#pragma unroll
            for (int sh = 0; sh < 2; ++sh)
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[sh] = fmaxf(mx[sh], p[sh][e]);
        }
        __builtin_amdgcn_s_waitcnt(0);
        exchange(mx);
        refer(mx);
        __syncthreads();
    }

    // whichever thread found it: barriers lie between
    if (threadIdx.x == 0 && holes != 0) raise_error(a.dev_error, SV_DEV_BAD_PAGE);

    // sums over the positions of a slot's lanes, and of the other wave
#pragma unroll
    for (int sh = 0; sh < 2; ++sh) {
        l[sh] += __shfl_xor(l[sh], 16);
        l[sh] += __shfl_xor(l[sh], 32);
        if (g == 0) tops[wave][sh * 16 + col] = l[sh];
    }
    __syncthreads();
#pragma unroll
    for (int sh = 0; sh < 2; ++sh) {
        const float o = tops[wave ^ 1][sh * 16 + col];
        l[sh] = half == 0 ? l[sh] + o : o + l[sh];
    }
    // the accumulators' slot is lane % 32: of either kind of lane the one's it is
    const int upper = lane >> 5;
    const bool odd16 = (lane >> 4) & 1;
    const float l_of = odd16 ? l[1] : l[0], m_of = odd16 ? m[1] : m[0];
    const int row_of = odd16 ? q_row[1] : q_row[0], head_of = odd16 ? head[1] : head[0];
    const bool live_of = odd16 ? live[1] : live[0];
    const int dim0 = half * (R / 2);
    if (!whole) {
        if (!live_of) return;
        const int64_t rec =
            (((int64_t)r * (a.k_max + 1) + row_of) * a.n_heads + head_of) * a.parts + part;
        float* o = a.part_out + rec * R + dim0 + 4 * upper;
#pragma unroll
        for (int i = 0; i < C::kDims; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *reinterpret_cast<f32x4*>(o + i * 32 + e * 8) =
                    f32x4{acc[i][4 * e], acc[i][4 * e + 1], acc[i][4 * e + 2], acc[i][4 * e + 3]};
        if (upper == 0 && half == 0) {
            a.part_ml[rec * 2] = m_of;
            a.part_ml[rec * 2 + 1] = l_of;
        }
        return;
    }
    // no weight at all: 0, also where 0 times a value was NaN
    const bool nothing = l_of == 0.0f;
    const float inv = nothing ? 0.0f : 1.0f / l_of;
    // eight dims a lane after the exchange of halves: an even or an odd eighth
    uint16_t* o = static_cast<uint16_t*>(a.out) + (int64_t)(lo + row_of) * a.out_ld +
                  (int64_t)head_of * R + dim0 + 8 * upper;
#pragma unroll
    for (int i = 0; i < C::kDims; ++i)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            uint32_t w[2][2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float x = acc[i][4 * (e + j) + 2 * n], y = acc[i][4 * (e + j) + 2 * n + 1];
                    // the mean first, then its scale: only their product has to be in range
                    w[j][n] = nothing ? 0u : pack_bf16(x * inv * kv_scale, y * inv * kv_scale);
                }
            const auto s0 = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
            const auto s1 = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
            if (live_of)
                *reinterpret_cast<uint4*>(o + i * 32 + e * 8) =
                    make_uint4(s0[0], s1[0], s0[1], s1[1]);
        }
    if (live_of && a.out_lse != nullptr && upper == 0 && half == 0)
        a.out_lse[(int64_t)(lo + row_of) * a.n_heads + head_of] =
            nothing ? -kInf : ((m_of - C::kHold) + log2f(l_of * exp2f(C::kHold))) * kLn2;
}

// Merges the parts of a (row, head): W waves, lanes over the dims, wave w the parts w,
// w + W, ...; the waves' sums meet in LDS, in a fixed order.  Bound by the latency of its
// loads: hipcc puts a part's behind the test that ends the sum, so that a wave has one on
// its way at a time (64 x 128 heads, 64 MB of parts: 13 us).
template <int R, bool F8, int W>
__global__ __launch_bounds__(256) void latent_join_kernel(LatentAttendArgs a) {
    constexpr int E = R / kWave;
    constexpr float kHold = Latent<R, F8>::kHold;
    __shared__ float factors[4][128];
    __shared__ float sums[W == 1 ? 1 : 4][R];
    const sv_latent_cache& c = a.cache;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, w0 = wave % W;
    const int per = (a.k_max + 1) * a.n_heads;
    const int64_t id = (int64_t)blockIdx.x * (4 / W) + wave / W;  // W = 4: of the workgroup
    if (id >= (int64_t)a.n_req * per) return;
    const int r = (int)(id / per), rest = (int)(id % per);
    const int row = rest / a.n_heads, head = rest % a.n_heads;
    const int lo = a.cu_rows[r], hi = a.cu_rows[r + 1], rows = hi - lo, ctx = a.ctx_len[r];
    if (lo < 0 || hi < lo || rows > a.k_max + 1 || hi > a.q_rows || row >= rows || ctx < 0 ||
        (int64_t)ctx + rows > (int64_t)a.max_pages * c.page_size)
        return;
    const int len = ctx + rows, plen = latent_part_len(len, a.parts, a.part_min);
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
    for (int p0 = w0; p0 < n; p0 += 4 * W) {
        float x[4][E];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) x[i][e] = po[(int64_t)min(p0 + i * W, n - 1) * R + e];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (p0 + i * W >= n) break;
            const float f = factor[p0 + i * W];
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] += f * x[i][e];
        }
    }
    if (W > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) sums[wave][lane * E + e] = o[e];
        __syncthreads();
        if (w0 != 0) return;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int i = lane * E + e;
            o[e] = (sums[0][i] + sums[1][i]) + (sums[2][i] + sums[3][i]);
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
    latent_kernel<R, F8><<<grid, 256, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.parts == 1) return e;
    const int64_t total = (int64_t)a.n_req * (a.k_max + 1) * a.n_heads;
    // few: a workgroup each, so that four parts are read at once
    if (total <= 2048) latent_join_kernel<R, F8, 4><<<(unsigned)total, 256, 0, stream>>>(a);
    else latent_join_kernel<R, F8, 1><<<(unsigned)((total + 3) / 4), 256, 0, stream>>>(a);
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
