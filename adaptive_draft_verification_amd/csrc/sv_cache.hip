// The paged key-value cache of the packed verify batch (gfx950, wave64):
// sv_cache_append writes a step's new keys and values behind each request's
// context, sv_cache_attend lets the packed rows attend to it.
#include "sv_device.h"
#include "sv_launch.h"
#include "sv_serve.h"

namespace sv {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_inff();

// ------------------------------------------------------------------- append

// One thread per 16 bytes of new keys or values.  Bound by its launch: 2 x
// rows x heads x dim values are read and written once.
template <bool F8>
__global__ void append_kernel(AppendArgs a) {
    const sv_cache& c = a.cache;
    const int chunks = c.head_dim / 8;
    const int64_t per_row = (int64_t)2 * c.n_kv_heads * chunks;
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= per_row * a.n_rows) return;
    const int row = (int)(i / per_row);
    int rest = (int)(i - (int64_t)row * per_row);
    const int ch = rest % chunks;
    rest /= chunks;
    const int h = rest % c.n_kv_heads;
    const bool is_v = rest >= c.n_kv_heads;
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
    const uint16_t* src = static_cast<const uint16_t*>(is_v ? a.v : a.k) + (int64_t)row * a.kv_ld +
                          h * c.head_dim + ch * 8;
    const uint4 w = *reinterpret_cast<const uint4*>(src);
    const int64_t at = (int64_t)page * c.page_stride + (int64_t)(t % c.page_size) * c.token_stride +
                       (int64_t)h * c.head_stride + ch * 8;
    if (!F8) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? c.v : c.k) + at) = w;
        return;
    }
    // x / scale rounded to fp32, then to e4m3 (nearest, ties to even), held
    // at the type's largest value; NaN stays NaN
    const float* scales = is_v ? c.v_scale : c.k_scale;
    const float s = scales != nullptr ? scales[h] : 1.0f;
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
    *reinterpret_cast<int2*>(static_cast<uint8_t*>(is_v ? c.v : c.k) + at) = make_int2(lo, hi);
}

// ------------------------------------------------------------------- attend
//
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

template <int D, bool F8, int MT, bool PG16>
__global__ __launch_bounds__(256, (Attend<D, F8, MT, PG16>::kOccupancy))
void attend_kernel(AttendArgs a) {
    using C = Attend<D, F8, MT, PG16>;
    __shared__ typename C::Smem sm;
    const sv_cache& c = a.cache;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    // grid: slot blocks fastest, then kv heads, requests and parts
    int id = spread(blockIdx.x, gridDim.x, a.xcd_run * a.slot_blocks);
    const int mb = id % a.slot_blocks;
    id /= a.slot_blocks;
    const int h = id % c.n_kv_heads;
    id /= c.n_kv_heads;
    int r = id % a.n_req;
    const int part = id / a.n_req;
    if (a.longest_first) r = longest(r, a.ctx_len, a.n_req, sm.lens);

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
    const int G = a.group;
    const int slots = rows * G - mb * 16 * MT;  // slots of this block
    if (slots <= 0) return;
    const int len = ctx + rows;
    const int plen = part_len(len, a.parts, a.part_min);
    const int begin = part * plen, end = min(len, begin + plen);
    if (begin >= len) return;
    const bool whole = plen >= len;  // the request's only part

    const char* kbase = static_cast<const char*>(c.k) + (int64_t)h * c.head_stride * C::kEsize;
    const char* vbase = static_cast<const char*>(c.v) + (int64_t)h * c.head_stride * C::kEsize;
    const int32_t* table = a.page_table + (int64_t)r * a.max_pages;
    // Byte offset of position t's row.  A bad page id is reported and its
    // positions count as absent (ok = false); the offset then is page 0's.
    auto row_offset = [&](int t, bool& ok) -> int64_t {
        t = min(t, len - 1);
        int page = table[t / c.page_size];
        ok = page >= 0 && page < c.n_pages;
        page = ok ? page : 0;
        return ((int64_t)page * c.page_stride + (int64_t)(t % c.page_size) * c.token_stride) *
               C::kEsize;
    };
    // Pages of a multiple of 16 positions hold each half of a tile (16
    // positions) in one page: two ids a tile, the same in every lane, fetched
    // a tile ahead of the loads that need them.
    const int last16 = (len - 1) & ~15;
    auto page_index = [&](int t) {
        return a.page_shift >= 0 ? t >> a.page_shift : (int)((unsigned)t / (unsigned)c.page_size);
    };
    struct Ids {
        int page[C::kHalves];
    };
    auto look_up = [&](int t0) {
        Ids p;
#pragma unroll
        for (int u = 0; u < C::kHalves; ++u)
            p.page[u] = table[page_index(min(t0 + 16 * u, last16))];
        return p;
    };

    Words<4> kr[C::kHalves][C::kKLoads];
    const int64_t tstride = c.token_stride * C::kEsize;
    const uint32_t koff = (uint32_t)(col * tstride) + g * 16;
    const uint32_t voff = (uint32_t)(g * 4 * tstride) + col * C::kDpl * C::kEsize;
    struct Values {
        Words<C::kVWords> r[4 * C::kHalves];
        uint32_t ok;  // bit j: the page of the lane's j-th position is good
    };
    Values vals;
    // Issues a tile's loads of keys or of values.
    auto load = [&](int t0, Ids ids, bool keys) __attribute__((always_inline)) {
        if (PG16) {
            const char* at[C::kHalves];
            uint32_t ok = 0;
#pragma unroll
            for (int u = 0; u < C::kHalves; ++u) {
                const int t = min(t0 + 16 * u, last16);
                int page = __builtin_amdgcn_readfirstlane(ids.page[u]);
                const bool good = page >= 0 && page < c.n_pages;
                ok |= good ? 0xfu << (4 * u) : 0u;
                page = good ? page : 0;
                const int slot = t - page_index(t) * c.page_size;
                const int64_t off =
                    ((int64_t)page * c.page_stride + (int64_t)slot * c.token_stride) * C::kEsize;
                at[u] = (keys ? kbase : vbase) + off;
            }
            if (keys) {
#pragma unroll
                for (int u = 0; u < C::kHalves; ++u)
#pragma unroll
                    for (int i = 0; i < C::kKLoads; ++i)
                        kr[u][i] = load_words<4>(at[u] + (koff + i * 64));
            } else {
                vals.ok = ok;
#pragma unroll
                for (int j = 0; j < 4 * C::kHalves; ++j)
                    vals.r[j] = load_words<C::kVWords>(at[j >> 2] +
                                                     (voff + (uint32_t)((j & 3) * tstride)));
            }
        } else if (keys) {
#pragma unroll
            for (int u = 0; u < C::kHalves; ++u) {
                bool ok;
                const char* at = kbase + row_offset(t0 + 16 * u + col, ok);
#pragma unroll
                for (int i = 0; i < C::kKLoads; ++i)
                    kr[u][i] = load_words<4>(at + (i * 64 + g * 16));
            }
        } else {
            vals.ok = 0;
#pragma unroll
            for (int j = 0; j < 4 * C::kHalves; ++j) {
                bool ok;
                const char* at = vbase + row_offset(t0 + 16 * (j >> 2) + g * 4 + (j & 3), ok);
                vals.ok |= ok ? 1u << j : 0u;
                vals.r[j] = load_words<C::kVWords>(at + col * C::kDpl * C::kEsize);
            }
        }
    };

    // the first tile's loads go out before anything else is done
    const int stride = C::kWaves * C::kTile;
    int t0 = begin + wave * C::kTile;
    Ids ids{};
    if (t0 < end) {
        if (PG16) ids = look_up(t0);
        load(t0, ids, true);
        load(t0, ids, false);
        if (PG16) ids = look_up(min(t0 + stride, len - 1));
    }

    // queries of the block's slots: wave w brings steps w, w + 4, ...
    const uint16_t* qp = static_cast<const uint16_t*>(a.q);
    int last[MT];  // the last position the lane's slot sees
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int i = mt * 16 + col, slot = mb * 16 * MT + i;
        const bool live = i < slots;
        const int row = slot / G, head = h * G + slot % G;
        last[mt] = live ? ctx + row : -1;
        for (int st = wave; st < C::kSteps; st += C::kWaves) {
            const int d = F8 ? (st / 2) * 64 + g * 16 + (st & 1) * 8 : st * 32 + g * 8;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (live)
                w = *reinterpret_cast<const uint4*>(qp + (int64_t)(lo + row) * a.q_ld +
                                                    (int64_t)head * D + d);
            sm.q[mt][st][lane] = w;
        }
    }
    __syncthreads();
    const float scale =
        a.scale * kLog2e * (F8 && c.k_scale != nullptr ? c.k_scale[h] : 1.0f);

    f32x4 acc[MT][C::kDpl];
    float m[MT], mu[MT], l[MT];  // running m (-inf: no score yet), the m used, sum
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int i = 0; i < C::kDpl; ++i) acc[mt][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        m[mt] = -kInf;
        mu[mt] = 0.0f;
        l[mt] = 0.0f;
    }
    int bad = 0;

    while (t0 < end) {
        constexpr int U = C::kHalves, J = 4 * U;  // halves; positions a lane holds
        constexpr uint32_t kAllOk = (1u << J) - 1;
        f32x4 s[MT][U];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int u = 0; u < U; ++u) s[mt][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int st = 0; st < C::kSteps; ++st) {
            bf16x8 k8[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (F8) {
                    const uint32_t w0 = kr[u][st / 2].w[(st & 1) * 2];
                    const uint32_t w1 = kr[u][st / 2].w[(st & 1) * 2 + 1];
                    k8[u] = as_bf16x8(e4m3_pair<false>(w0), e4m3_pair<true>(w0),
                                      e4m3_pair<false>(w1), e4m3_pair<true>(w1));
                } else {
                    const Words<4>& w = kr[u][F8 ? 0 : st];
                    k8[u] = as_bf16x8(w.w[0], w.w[1], w.w[2], w.w[3]);
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const uint4 w = sm.q[mt][st][lane];
                const bf16x8 q8 = as_bf16x8(w.x, w.y, w.z, w.w);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    s[mt][u] =
                        __builtin_amdgcn_mfma_f32_16x16x32_bf16(k8[u], q8, s[mt][u], 0, 0, 0);
            }
        }
        // the next tile's keys, in flight over the softmax and the product with
        // the values (the scores are taken first: the keys' registers); its
        // values follow the product, into the same registers.  A second set of
        // value registers spills: 445 us of 256 requests against 394.
        const int t1 = t0 + stride;
        const bool more = t1 < end;
        const Ids ids1 = ids;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int u = 0; u < U; ++u) asm volatile("" : "+v"(s[mt][u]));
        if (more) {
            load(t1, ids1, true);
            if (PG16) ids = look_up(min(t1 + stride, len - 1));
        }
        __builtin_amdgcn_sched_barrier(0);

        // Positions past the context are not seen by every row; positions past
        // the end, or on a bad page, by none: their values are zeroed, since 0
        // times what lies there may be NaN.  A value that is not finite behind
        // the context poisons the product for the rows that do not see it.
        if (vals.ok != kAllOk) bad = 1;
        const bool edge = t0 + C::kTile > ctx || __ballot(vals.ok != kAllOk) != 0;
        bool poison = false;
        if (edge) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int t = t0 + 16 * (j >> 2) + g * 4 + (j & 3);
                const bool in = t < len && ((vals.ok >> j) & 1);
                bool nf = false;
#pragma unroll
                for (int i = 0; i < C::kVWords; ++i) {
                    if (!in) vals.r[j].w[i] = 0;
                    if (F8) {
                        nf |= bf16_pair_nonfinite(e4m3_pair<false>(vals.r[j].w[i])) ||
                              bf16_pair_nonfinite(e4m3_pair<true>(vals.r[j].w[i]));
                    } else {
                        nf |= bf16_pair_nonfinite(vals.r[j].w[i]);
                    }
                }
                poison |= nf && t > ctx;
            }
            poison = __ballot(poison) != 0;
        }
        bf16x8 pb[MT], pr[MT];  // the weights' upper halves and rests
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            if (mt * 16 >= slots) break;
            float p[J];
#pragma unroll
            for (int j = 0; j < J; ++j) p[j] = s[mt][j >> 2][j & 3] * scale;
            if (edge) {
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int t = t0 + 16 * (j >> 2) + g * 4 + (j & 3);
                    if (t > last[mt] || !((vals.ok >> j) & 1)) p[j] = -kInf;
                }
            }
            float mx = p[0];
#pragma unroll
            for (int j = 1; j < J; ++j) mx = fmaxf(mx, p[j]);
            // m moves only when a score passes the maximum it came from by 2^8,
            // or the sum is full: sums and outputs are relative to it either
            // way; most tiles then rescale nothing
            if (__ballot(mx > m[mt] + (8.0f - C::kHold) || (!F8 && l[mt] > C::kFull)) != 0) {
                mx = fmaxf(mx, __shfl_xor(mx, 16));
                mx = fmaxf(mx, __shfl_xor(mx, 32));
                float to = fmaxf(m[mt], mx + C::kHold);
                if (!F8) {
                    float most = fmaxf(l[mt], __shfl_xor(l[mt], 16));
                    most = fmaxf(most, __shfl_xor(most, 32));
                    if (most > C::kFull) to += C::kRaise;
                }
                if (to > m[mt]) {
                    const float f = fast_exp2(m[mt] - to);  // m = -inf: 0
#pragma unroll
                    for (int i = 0; i < C::kDpl; ++i) acc[mt][i] *= f;
                    l[mt] *= f;
                    m[mt] = mu[mt] = to;
                }
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                p[j] = fast_exp2(p[j] - mu[mt]);
                l[mt] += p[j];
            }
            // Weights go into the matrix product as two bf16 terms, the upper
            // half of the fp32 weight and the rest, off by at most 2^-15 of each.
            // Both are positive where the weight is (the rest of 1 + 2^-23 times
            // it is taken): an infinite value times 0 or a negative rest would
            // make NaN.  One term (2^-8) let the error against 64 bits grow by up
            // to a quarter; the second costs 0 .. 2 % where reading bounds the
            // call (256 requests, ctx 4096: 392.0 and 393.7 us; 3 x 100,005 e4m3:
            // 141.4 and 144.8), 8 % at four slot tiles.
            constexpr float kOneUp = 1.0f + 0x1p-23f;
            uint32_t hw[4], rw[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a = __float_as_uint(p[2 * i]), b = __float_as_uint(p[2 * i + 1]);
                hw[i] = __builtin_amdgcn_perm(b, a, 0x07060302u);
                rw[i] = pack_bf16(fmaf(p[2 * i], kOneUp, -bf16_hi(a)),
                                  fmaf(p[2 * i + 1], kOneUp, -bf16_hi(b)));
            }
            pb[mt] = as_bf16x8(hw[0], hw[1], hw[2], hw[3]);
            pr[mt] = as_bf16x8(rw[0], rw[1], rw[2], rw[3]);
            if (poison) {
                // position by position, each row only what it sees
                for (int gg = 0; gg < 4; ++gg) {
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        const float pj = __shfl(p[j], gg * 16 + col);
                        const int t = t0 + 16 * (j >> 2) + gg * 4 + (j & 3);
                        bool ok;
                        const char* at = vbase + row_offset(t, ok) + g * C::kAcc * C::kEsize;
                        if (t > last[mt] || t >= len || !ok) continue;
#pragma unroll
                        for (int e = 0; e < C::kAcc; ++e) {
                            float v;
                            if (F8) {
                                const uint32_t w = reinterpret_cast<const uint8_t*>(at)[e];
                                v = __uint_as_float(e4m3_pair<false>(w) << 16);
                            } else {
                                v = __uint_as_float(
                                    (uint32_t)reinterpret_cast<const uint16_t*>(at)[e] << 16);
                            }
                            acc[mt][e % C::kDpl][e / C::kDpl] += pj * v;
                        }
                    }
                }
            }
        }
        if (!poison) {
#pragma unroll
            for (int i2 = 0; i2 < C::kDpl / 2; ++i2) {
                uint32_t w[8];  // dims 2 i2 and 2 i2 + 1 of the lane's 8 positions
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const Words<C::kVWords>& v = vals.r[j];
                    if (F8)
                        w[j] = (i2 & 1) ? e4m3_pair<true>(v.w[i2 / 2])
                                        : e4m3_pair<false>(v.w[i2 / 2]);
                    else
                        w[j] = v.w[F8 ? 0 : i2];
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t sel = half ? 0x07060302u : 0x05040100u;
                    const bf16x8 vt = as_bf16x8(__builtin_amdgcn_perm(w[1], w[0], sel),
                                                __builtin_amdgcn_perm(w[3], w[2], sel),
                                                __builtin_amdgcn_perm(w[5], w[4], sel),
                                                __builtin_amdgcn_perm(w[7], w[6], sel));
                    const int i = 2 * i2 + half;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        if (mt * 16 >= slots) break;
                        acc[mt][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt, pb[mt],
                                                                             acc[mt][i], 0, 0, 0);
                        acc[mt][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt, pr[mt],
                                                                             acc[mt][i], 0, 0, 0);
                    }
                }
            }
        }
        if (more) load(t1, ids1, false);
        t0 = t1;
    }
    if (__ballot(bad) != 0 && lane == 0) raise_error(a.dev_error, SV_DEV_BAD_PAGE);

    // sums over the four lane groups of a slot
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        l[mt] += __shfl_xor(l[mt], 16);
        l[mt] += __shfl_xor(l[mt], 32);
    }
    // the waves' results, two by two: 2, 3 into 0, 1, then 1 into 0
#pragma unroll
    for (int round = 0; round < 2; ++round) {
        const int from = round == 0 ? 2 : 1, n = round == 0 ? 2 : 1;
        __syncthreads();
        if (wave >= from && wave < from + n) {
            const int b = wave - from;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if (mt * 16 >= slots) break;
#pragma unroll
                for (int i = 0; i < C::kDpl; ++i)
                    *reinterpret_cast<f32x4*>(sm.part.acc[b][mt][i][lane]) = acc[mt][i];
                sm.part.m[b][mt][lane] = m[mt];
                sm.part.l[b][mt][lane] = l[mt];
            }
        }
        __syncthreads();
        if (wave < n) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if (mt * 16 >= slots) break;
                const float m2 = sm.part.m[wave][mt][lane], l2 = sm.part.l[wave][mt][lane];
                const float mx = fmaxf(m[mt], m2);
                const float f1 = m[mt] == mx ? 1.0f : fast_exp2(m[mt] - mx);
                const float f2 = m2 == mx ? 1.0f : fast_exp2(m2 - mx);
                l[mt] = l[mt] * f1 + l2 * f2;
                m[mt] = mx;
#pragma unroll
                for (int i = 0; i < C::kDpl; ++i) {
                    const f32x4 o = *reinterpret_cast<const f32x4*>(sm.part.acc[wave][mt][i][lane]);
                    acc[mt][i] = acc[mt][i] * f1 + o * f2;
                }
            }
        }
    }
    if (wave != 0) return;

    const float vscale = F8 && c.v_scale != nullptr ? c.v_scale[h] : 1.0f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int i = mt * 16 + col, slot = mb * 16 * MT + i;
        if (i >= slots) continue;
        const int row = slot / G, head = h * G + slot % G;
        if (whole) {
            // no weight at all: 0, also where 0 times a value was NaN
            if (l[mt] == 0.0f) {
#pragma unroll
                for (int e = 0; e < C::kDpl; ++e) acc[mt][e] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            }
            // the mean first, then its scale: only their product has to be in range
            const float inv = l[mt] == 0.0f ? 0.0f : 1.0f / l[mt];
            uint32_t w[C::kAcc / 2];
#pragma unroll
            for (int e = 0; e < C::kAcc; e += 2)
                w[e / 2] =
                    pack_bf16(acc[mt][e % C::kDpl][e / C::kDpl] * inv * vscale,
                              acc[mt][(e + 1) % C::kDpl][(e + 1) / C::kDpl] * inv * vscale);
            uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) +
                                                (int64_t)(lo + row) * a.out_ld +
                                                (int64_t)head * D + g * C::kAcc);
#pragma unroll
            for (int e = 0; e < C::kAcc / 8; ++e)
                o[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
            if (a.out_lse != nullptr && g == 0)
                a.out_lse[(int64_t)(lo + row) * a.n_heads + head] =
                    l[mt] == 0.0f
                        ? -kInf
                        : ((m[mt] - C::kHold) + log2f(l[mt] * exp2f(C::kHold))) * kLn2;
        } else {
            const int64_t rec = (((int64_t)r * a.n_heads + head) * (a.k_max + 1) + row) * a.parts +
                                part;
            f32x4* o = reinterpret_cast<f32x4*>(a.part_out + rec * D + g * C::kAcc);
#pragma unroll
            for (int e = 0; e < C::kAcc; e += 4) {
                f32x4 x;
#pragma unroll
                for (int i4 = 0; i4 < 4; ++i4)
                    x[i4] = acc[mt][(e + i4) % C::kDpl][(e + i4) / C::kDpl];
                o[e / 4] = x;
            }
            if (g == 0) {
                a.part_ml[rec * 2] = m[mt];
                a.part_ml[rec * 2 + 1] = l[mt];
            }
        }
    }
}

// Merges the parts of a (row, head): W waves, wave w the parts w, w + W, ...
// (eight loads in flight each), lanes over the dims; the waves' sums meet in
// LDS, in a fixed order.  A request of one part wrote its outputs itself.
template <int D, bool F8, int W>
__global__ __launch_bounds__(256) void join_kernel(AttendArgs a) {
    constexpr int E = D / 64, kEach = 4 / W;  // (row, head)s a workgroup takes at once
    constexpr float kHold = Attend<D, F8, 1, true>::kHold;
    __shared__ float sm_o[4][D], sm_f[4][128];
    const sv_cache& c = a.cache;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int w = wave % W;
    const int per = (a.k_max + 1) * a.n_heads;
    const int64_t total = (int64_t)a.n_req * per;
    for (int64_t first = (int64_t)blockIdx.x * kEach; first < total;
         first += (int64_t)gridDim.x * kEach) {
        const int64_t id = first + wave / W;
        const int r = (int)(min(id, total - 1) / per), rest = (int)(min(id, total - 1) % per);
        const int row = rest / a.n_heads, head = rest % a.n_heads;
        const int lo = a.cu_rows[r], hi = a.cu_rows[r + 1], rows = hi - lo, ctx = a.ctx_len[r];
        bool live = id < total && lo >= 0 && hi >= lo && rows <= a.k_max + 1 && hi <= a.q_rows &&
                    row < rows && ctx >= 0 &&
                    (int64_t)ctx + rows <= (int64_t)a.max_pages * c.page_size;
        const int len = ctx + rows, plen = live ? part_len(len, a.parts, a.part_min) : 1;
        live = live && plen < len;
        if (W == 4 && !live) continue;  // the same in every wave
        const int n = live ? (len + plen - 1) / plen : 0;  // at most 128
        const int64_t rec =
            (((int64_t)r * a.n_heads + head) * (a.k_max + 1) + row) * a.parts;
        const float* ml = a.part_ml + rec * 2;
        const float* po = a.part_out + rec * D + lane * E;
        float m = -kInf, l = 0.0f, o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.0f;
        if (live) {
            // every wave: the largest maximum and the parts' factors, two a lane
            float m0 = -kInf, m1 = -kInf, l0 = 0.0f, l1 = 0.0f;
            if (lane < n) m0 = ml[2 * lane], l0 = ml[2 * lane + 1];
            if (lane + 64 < n) m1 = ml[2 * lane + 128], l1 = ml[2 * lane + 129];
            m = wave_max(fmaxf(m0, m1));
            const float f0 = m0 == m ? 1.0f : fast_exp2(m0 - m);
            const float f1 = m1 == m ? 1.0f : fast_exp2(m1 - m);
            l = wave_sum((lane < n ? f0 * l0 : 0.0f) + (lane + 64 < n ? f1 * l1 : 0.0f));
            // over the whole sum before the outputs are added up: they are then
            // shares of the mean, and stay in range
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            float* factor = sm_f[wave];
            factor[lane] = f0 * inv;
            factor[lane + 64] = f1 * inv;
            __builtin_amdgcn_wave_barrier();
            for (int p0 = w; p0 < n; p0 += 8 * W) {
                float x[8][E];
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        x[i][e] = po[(int64_t)min(p0 + W * i, n - 1) * D + e];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (p0 + W * i >= n) break;
                    const float f = factor[p0 + W * i];
#pragma unroll
                    for (int e = 0; e < E; ++e) o[e] += f * x[i][e];
                }
            }
        }
        if (W > 1) {
#pragma unroll
            for (int e = 0; e < E; ++e) sm_o[wave][lane * E + e] = o[e];
            __syncthreads();
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int i = lane * E + e;
                o[e] = (sm_o[0][i] + sm_o[1][i]) + (sm_o[2][i] + sm_o[3][i]);
            }
            __syncthreads();
        }
        if (!live || w != 0) continue;
        const float vscale = F8 && c.v_scale != nullptr ? c.v_scale[head / a.group] : 1.0f;
        uint16_t* out = static_cast<uint16_t*>(a.out) + (int64_t)(lo + row) * a.out_ld +
                        (int64_t)head * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e)
            out[e] = (uint16_t)pack_bf16(l == 0.0f ? 0.0f : o[e] * vscale, 0.0f);
        if (a.out_lse != nullptr && lane == 0)
            a.out_lse[(int64_t)(lo + row) * a.n_heads + head] =
                l == 0.0f ? -kInf : ((m - kHold) + log2f(l * exp2f(kHold))) * kLn2;
    }
}

template <int D, bool F8>
void run_join(const AttendArgs& a, hipStream_t stream) {
    const int64_t total = (int64_t)a.n_req * (a.k_max + 1) * a.n_heads;
    // up to 16 parts one wave keeps them all in flight in two goes
    if (a.parts <= 16) {
        const int64_t grid = (total + 3) / 4;
        join_kernel<D, F8, 1><<<(unsigned)(grid < 4096 ? grid : 4096), 256, 0, stream>>>(a);
    } else {
        join_kernel<D, F8, 4><<<(unsigned)(total < 4096 ? total : 4096), 256, 0, stream>>>(a);
    }
}

template <int D, bool F8, int MT>
void run_attend(const AttendArgs& a, unsigned grid, hipStream_t stream) {
    if (a.cache.page_size % 16 == 0 && 16 * a.cache.token_stride <= (int64_t)1 << 28)
        attend_kernel<D, F8, MT, true><<<grid, 256, 0, stream>>>(a);
    else
        attend_kernel<D, F8, MT, false><<<grid, 256, 0, stream>>>(a);
}

template <int D, bool F8>
hipError_t run_attend_mt(const AttendArgs& a, hipStream_t stream) {
    const unsigned grid =
        (unsigned)((int64_t)a.cache.n_kv_heads * a.n_req * a.slot_blocks * a.parts);
    if (a.slot_tiles == 1) run_attend<D, F8, 1>(a, grid, stream);
    else if constexpr (D == 256) return hipErrorInvalidValue;  // AttendPlan takes one
    else if (a.slot_tiles == 2) run_attend<D, F8, 2>(a, grid, stream);
    else run_attend<D, F8, 4>(a, grid, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.parts == 1) return e;
    run_join<D, F8>(a, stream);
    return hipGetLastError();
}

template <int D>
hipError_t run_attend_d(const AttendArgs& a, hipStream_t stream) {
    return a.cache.dtype == SV_E4M3 ? run_attend_mt<D, true>(a, stream)
                                    : run_attend_mt<D, false>(a, stream);
}

}  // namespace

hipError_t launch_cache_append(const AppendArgs& a, hipStream_t stream) {
    const int64_t threads =
        (int64_t)a.n_rows * 2 * a.cache.n_kv_heads * (a.cache.head_dim / 8);
    const unsigned grid = (unsigned)((threads + 255) / 256);
    if (a.cache.dtype == SV_E4M3)
        append_kernel<true><<<grid, 256, 0, stream>>>(a);
    else
        append_kernel<false><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_cache_attend(const AttendArgs& a, hipStream_t stream) {
    switch (a.cache.head_dim) {
        case 64: return run_attend_d<64>(a, stream);
        case 128: return run_attend_d<128>(a, stream);
        default: return run_attend_d<256>(a, stream);
    }
}

}  // namespace sv
