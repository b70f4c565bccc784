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
    static constexpr int kTile = 32;        // positions a wave takes at once
    static constexpr int kWaves = 4;
    static constexpr int kSteps = D / 32;   // products a 16-position score needs
    static constexpr int kKLoads = F8 ? D / 64 : D / 32;  // 16-byte loads of a key row's share
    static constexpr int kDpl = D / 16;     // dims a lane loads of a value row
    static constexpr int kVWords = F8 ? kDpl / 4 : kDpl / 2;
    static constexpr int kAcc = D / 4;      // accumulators a slot tile and lane
    static constexpr int kEsize = F8 ? 1 : 2;

    // Partial result of a slot tile in one lane: running maximum (in units of
    // log2), sum and unnormalised output of slot lane % 16.
    struct Smem {
        float acc[2][MT][kAcc / 4][kWave][4];
        float m[2][MT][kWave], l[2][MT][kWave];
    };
};

template <int D, bool F8, int MT, bool PG16>
__global__ __launch_bounds__(256) void attend_kernel(AttendArgs a) {
    using C = Attend<D, F8, MT, PG16>;
    __shared__ typename C::Smem sm;
    const sv_cache& c = a.cache;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 15, g = lane >> 4;
    // grid: kv heads fastest, then requests, slot blocks and parts
    int id = blockIdx.x;
    const int h = id % c.n_kv_heads;
    id /= c.n_kv_heads;
    const int r = id % a.n_req;
    id /= a.n_req;
    const int mb = id % a.slot_blocks, part = id / a.slot_blocks;

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
    const int plen = part_len(len, a.parts);
    const int begin = part * plen, end = min(len, begin + plen);
    if (begin >= len) return;

    // queries of this lane's slot, as operand B
    bf16x8 q[MT][C::kSteps];
    int last[MT];  // the last position the slot sees
    const uint16_t* qp = static_cast<const uint16_t*>(a.q);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int i = mt * 16 + col, slot = mb * 16 * MT + i;
        const bool live = i < slots;
        const int row = slot / G, head = h * G + slot % G;
        last[mt] = live ? ctx + row : -1;
#pragma unroll
        for (int s = 0; s < C::kSteps; ++s) {
            const int d = F8 ? (s / 2) * 64 + g * 16 + (s & 1) * 8 : s * 32 + g * 8;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (live)
                w = *reinterpret_cast<const uint4*>(qp + (int64_t)(lo + row) * a.q_ld +
                                                    (int64_t)head * D + d);
            q[mt][s] = as_bf16x8(w.x, w.y, w.z, w.w);
        }
    }
    const float scale =
        a.scale * kLog2e * (F8 && c.k_scale != nullptr ? c.k_scale[h] : 1.0f);

    f32x4 acc[MT][C::kDpl];
    float m[MT], mu[MT], l[MT];  // running max (-inf: none yet), the max used, sum
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int i = 0; i < C::kDpl; ++i) acc[mt][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        m[mt] = -kInf;
        mu[mt] = 0.0f;
        l[mt] = 0.0f;
    }

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

    // The byte offsets of a tile's rows: pages of a multiple of 16 positions
    // hold each half of a tile (16 positions) in one page.
    struct Rows {
        int64_t half[2];
        bool ok[2];
    };
    auto find = [&](int t0) {
        Rows p;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int t = min(t0 + 16 * s, (len - 1) & ~15);
            int page = table[t / c.page_size];
            p.ok[s] = page >= 0 && page < c.n_pages;
            page = p.ok[s] ? page : 0;
            p.half[s] = ((int64_t)page * c.page_stride +
                         (int64_t)(t % c.page_size) * c.token_stride) * C::kEsize;
        }
        return p;
    };

    Words<4> kr[2][C::kKLoads];
    Words<C::kVWords> vr[8];
    uint32_t vok = 0;  // bit j: the page of the lane's j-th position is good
    const int64_t tstride = c.token_stride * C::kEsize;
    auto load_k = [&](int t0, const Rows& p) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const char* at;
            if (PG16) {
                at = kbase + p.half[s] + col * tstride;
            } else {
                bool ok;
                at = kbase + row_offset(t0 + 16 * s + col, ok);
            }
#pragma unroll
            for (int i = 0; i < C::kKLoads; ++i) kr[s][i] = load_words<4>(at + (i * 64 + g * 16));
        }
    };
    auto load_v = [&](int t0, const Rows& p) {
        vok = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int s = j >> 2, o = g * 4 + (j & 3);
            const char* at;
            bool ok;
            if (PG16) {
                at = vbase + p.half[s] + o * tstride;
                ok = p.ok[s];
            } else {
                at = vbase + row_offset(t0 + 16 * s + o, ok);
            }
            vok |= ok ? 1u << j : 0u;
            vr[j] = load_words<C::kVWords>(at + col * C::kDpl * C::kEsize);
        }
    };

    const int stride = C::kWaves * C::kTile;
    int t0 = begin + wave * C::kTile;
    int bad = 0;
    for (; t0 < end; t0 += stride) {
        Rows rows_at{};
        if (PG16) rows_at = find(t0);
        load_k(t0, rows_at);
        load_v(t0, rows_at);
        // the values' rows of the 8 positions, as bf16 pairs of dims
        uint32_t vw[8][C::kDpl / 2];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
            for (int i = 0; i < C::kVWords; ++i) {
                if (F8) {
                    vw[j][2 * i] = e4m3_pair<false>(vr[j].w[i]);
                    vw[j][2 * i + 1] = e4m3_pair<true>(vr[j].w[i]);
                } else {
                    vw[j][i] = vr[j].w[i];
                }
            }
        }
        if (vok != 0xffu) bad = 1;
        // positions past the context are not seen by every row; positions
        // past the end, or on a bad page, by none: their values are zeroed,
        // since 0 times what lies there may be NaN
        const bool edge = t0 + C::kTile > ctx || __ballot(vok != 0xffu) != 0;
        bool poison = false;
        if (edge) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int t = t0 + 16 * (j >> 2) + g * 4 + (j & 3);
                const bool in = t < len && ((vok >> j) & 1);
                bool nf = false;
#pragma unroll
                for (int i = 0; i < C::kDpl / 2; ++i) {
                    if (!in) vw[j][i] = 0;
                    nf |= bf16_pair_nonfinite(vw[j][i]);
                }
                poison |= nf && t > ctx;
            }
            poison = __ballot(poison) != 0;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            if (mt * 16 >= slots) break;
            f32x4 s[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                s[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int st = 0; st < C::kSteps; ++st) {
                    bf16x8 k8;
                    if (F8) {
                        const uint32_t w0 = kr[u][st / 2].w[(st & 1) * 2];
                        const uint32_t w1 = kr[u][st / 2].w[(st & 1) * 2 + 1];
                        k8 = as_bf16x8(e4m3_pair<false>(w0), e4m3_pair<true>(w0),
                                       e4m3_pair<false>(w1), e4m3_pair<true>(w1));
                    } else {
                        const Words<4>& w = kr[u][st];
                        k8 = as_bf16x8(w.w[0], w.w[1], w.w[2], w.w[3]);
                    }
                    s[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k8, q[mt][st], s[u], 0, 0, 0);
                }
            }
            float p[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) p[j] = s[j >> 2][j & 3] * scale;
            if (edge) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int t = t0 + 16 * (j >> 2) + g * 4 + (j & 3);
                    if (t > last[mt] || !((vok >> j) & 1)) p[j] = -kInf;
                }
            }
            float mx = p[0];
#pragma unroll
            for (int j = 1; j < 8; ++j) mx = fmaxf(mx, p[j]);
            // the maximum moves only when a score passes it by 2^8: sums and
            // outputs are relative to it either way, and stay far from
            // overflow; most tiles then rescale nothing
            if (__ballot(mx > m[mt] + 8.0f) != 0) {
                mx = fmaxf(mx, __shfl_xor(mx, 16));
                mx = fmaxf(mx, __shfl_xor(mx, 32));
                if (mx > m[mt]) {
                    const float f = fast_exp2(m[mt] - mx);  // m = -inf: 0
#pragma unroll
                    for (int i = 0; i < C::kDpl; ++i) acc[mt][i] *= f;
                    l[mt] *= f;
                    m[mt] = mu[mt] = mx;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                p[j] = fast_exp2(p[j] - mu[mt]);
                l[mt] += p[j];
            }
            if (poison) {
                // a later row's value is not finite: no product over all 32
                // positions (0 times it is NaN); position by position instead
                for (int gg = 0; gg < 4; ++gg) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
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
                continue;
            }
            // weights rounded to bf16 for the matrix product: at most 2^-9 of
            // each, as far as the output's own rounding
            const bf16x8 pb = as_bf16x8(pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]),
                                        pack_bf16(p[4], p[5]), pack_bf16(p[6], p[7]));
#pragma unroll
            for (int i = 0; i < C::kDpl; ++i) {
                const uint32_t sel = (i & 1) ? 0x07060302u : 0x05040100u;
                const bf16x8 vt = as_bf16x8(
                    __builtin_amdgcn_perm(vw[1][i / 2], vw[0][i / 2], sel),
                    __builtin_amdgcn_perm(vw[3][i / 2], vw[2][i / 2], sel),
                    __builtin_amdgcn_perm(vw[5][i / 2], vw[4][i / 2], sel),
                    __builtin_amdgcn_perm(vw[7][i / 2], vw[6][i / 2], sel));
                acc[mt][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt, pb, acc[mt][i], 0, 0, 0);
            }
        }
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
                    *reinterpret_cast<f32x4*>(sm.acc[b][mt][i][lane]) = acc[mt][i];
                sm.m[b][mt][lane] = m[mt];
                sm.l[b][mt][lane] = l[mt];
            }
        }
        __syncthreads();
        if (wave < n) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if (mt * 16 >= slots) break;
                const float m2 = sm.m[wave][mt][lane], l2 = sm.l[wave][mt][lane];
                const float mx = fmaxf(m[mt], m2);
                const float f1 = m[mt] == mx ? 1.0f : fast_exp2(m[mt] - mx);
                const float f2 = m2 == mx ? 1.0f : fast_exp2(m2 - mx);
                l[mt] = l[mt] * f1 + l2 * f2;
                m[mt] = mx;
#pragma unroll
                for (int i = 0; i < C::kDpl; ++i) {
                    const f32x4 o = *reinterpret_cast<const f32x4*>(sm.acc[wave][mt][i][lane]);
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
        if (a.parts == 1) {
            const float inv = l[mt] == 0.0f ? 0.0f : vscale / l[mt];
            uint32_t w[C::kAcc / 2];
#pragma unroll
            for (int e = 0; e < C::kAcc; e += 2)
                w[e / 2] = pack_bf16(acc[mt][e % C::kDpl][e / C::kDpl] * inv,
                                     acc[mt][(e + 1) % C::kDpl][(e + 1) / C::kDpl] * inv);
            uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) +
                                                (int64_t)(lo + row) * a.out_ld +
                                                (int64_t)head * D + g * C::kAcc);
#pragma unroll
            for (int e = 0; e < C::kAcc / 8; ++e)
                o[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
            if (a.out_lse != nullptr && g == 0)
                a.out_lse[(int64_t)(lo + row) * a.n_heads + head] =
                    l[mt] == 0.0f ? -kInf : (m[mt] + log2f(l[mt])) * kLn2;
        } else {
            const int64_t rec = (((int64_t)r * a.n_heads + head) * (a.k_max + 1) + row) * a.parts +
                                part;
            float* o = a.part_out + rec * D + g * C::kAcc;
#pragma unroll
            for (int e = 0; e < C::kAcc; ++e) o[e] = acc[mt][e % C::kDpl][e / C::kDpl] * vscale;
            if (g == 0) {
                a.part_ml[rec * 2] = m[mt];
                a.part_ml[rec * 2 + 1] = l[mt];
            }
        }
    }
}

// Merges the parts of one (row, head): one wave, lanes over the dims.
template <int D>
__global__ __launch_bounds__(256) void join_kernel(AttendArgs a) {
    const sv_cache& c = a.cache;
    const int lane = threadIdx.x & 63;
    const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int per = (a.k_max + 1) * a.n_heads;
    if (id >= (int64_t)a.n_req * per) return;
    const int r = (int)(id / per), rest = (int)(id % per);
    const int head = rest / (a.k_max + 1), row = rest % (a.k_max + 1);
    const int lo = a.cu_rows[r], hi = a.cu_rows[r + 1], rows = hi - lo, ctx = a.ctx_len[r];
    if (lo < 0 || hi < lo || rows > a.k_max + 1 || hi > a.q_rows || row >= rows) return;
    if (ctx < 0 || (int64_t)ctx + rows > (int64_t)a.max_pages * c.page_size) return;
    const int len = ctx + rows, plen = part_len(len, a.parts);
    const int n = (len + plen - 1) / plen;
    const int64_t rec = (((int64_t)r * a.n_heads + head) * (a.k_max + 1) + row) * a.parts;
    float m = -kInf;
    for (int p = 0; p < n; ++p) m = fmaxf(m, a.part_ml[(rec + p) * 2]);
    float l = 0.0f, o[D / 64];
#pragma unroll
    for (int e = 0; e < D / 64; ++e) o[e] = 0.0f;
    for (int p = 0; p < n; ++p) {
        const float mp = a.part_ml[(rec + p) * 2];
        const float f = mp == m ? 1.0f : fast_exp2(mp - m);
        l += f * a.part_ml[(rec + p) * 2 + 1];
        const float* src = a.part_out + (rec + p) * D + lane * (D / 64);
#pragma unroll
        for (int e = 0; e < D / 64; ++e) o[e] += f * src[e];
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t* out = static_cast<uint16_t*>(a.out) + (int64_t)(lo + row) * a.out_ld +
                    (int64_t)head * D + lane * (D / 64);
#pragma unroll
    for (int e = 0; e < D / 64; ++e) out[e] = (uint16_t)pack_bf16(o[e] * inv, 0.0f);
    if (a.out_lse != nullptr && lane == 0)
        a.out_lse[(int64_t)(lo + row) * a.n_heads + head] =
            l == 0.0f ? -kInf : (m + log2f(l)) * kLn2;
}

template <int D, bool F8, int MT>
void run_attend(const AttendArgs& a, unsigned grid, hipStream_t stream) {
    if (a.cache.page_size % 16 == 0)
        attend_kernel<D, F8, MT, true><<<grid, 256, 0, stream>>>(a);
    else
        attend_kernel<D, F8, MT, false><<<grid, 256, 0, stream>>>(a);
}

template <int D, bool F8>
hipError_t run_attend_mt(const AttendArgs& a, hipStream_t stream) {
    const unsigned grid =
        (unsigned)((int64_t)a.cache.n_kv_heads * a.n_req * a.slot_blocks * a.parts);
    if (a.slot_tiles == 1) run_attend<D, F8, 1>(a, grid, stream);
    else if (a.slot_tiles == 2) run_attend<D, F8, 2>(a, grid, stream);
    else if constexpr (D < 256) run_attend<D, F8, 4>(a, grid, stream);
    else return hipErrorInvalidValue;
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.parts == 1) return e;
    const int64_t waves = (int64_t)a.n_req * (a.k_max + 1) * a.n_heads;
    join_kernel<D><<<(unsigned)((waves + 3) / 4), 256, 0, stream>>>(a);
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
