// The truncated law of a logit row (gfx950, wave64): which ids a request's
// temperature, top-k, top-p and min-p leave, and their weights.
//
// With m the row's largest logit and T the temperature, w(x) =
// exp((z(x) - m) / T).  Ids are ordered by logit, larger first, ties to the
// lower id (-0 equals 0, -inf takes no part).  The support is the prefix of
// that order that top-k (k ids), top-p (the fewest ids whose weight reaches p
// of the first k's) and min-p (weights >= s) all leave; T = 0 leaves one id.
//
// Weights, sums and borders are taken in 64 bits: with 10^5 ids a cumulative
// sum in 32 bits puts a border or a drawn id one off in every few rows, and a
// draw would depend on how the sum was split.  Sums that atomics gather are
// fixed-point integers (two 64-bit words, 43 bits each below the point), so
// their order does not change them.
//
// One workgroup of 1024 threads holds a row.  What takes part in the search
// for the border is first cut down by a bound that costs one pass (the k-th
// largest of the threads' own maxima, min-p's logit, or the logit below which
// all ids together weigh less than top-p leaves out); what is left is kept in
// LDS if it fits, and the search goes over that list instead of the row.  The
// border is found digit by digit: 256 bins over 8 bits of the ordered key, the
// bin that holds the border, then the next 8 bits within it.
#pragma once

#include "sv_device.h"
#include "sv_serve.h"

namespace sv {
namespace law {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kList = 2048;  // candidates kept in LDS
constexpr float kInf = __builtin_inff();
constexpr uint32_t kMinusInfKey = 0x007fffffu;

// Ascending in the logit; -0 and 0 alike.
__device__ __forceinline__ uint32_t order_key(float z) {
    const uint32_t b = __float_as_uint(z + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// A fixed-point mass: hi 2^-43 + lo 2^-86, each weight at most 1, 2^20 of them.
struct Mass {
    unsigned long long hi, lo;
    __device__ __forceinline__ double value() const {
        return (double)hi * 0x1p-43 + (double)lo * 0x1p-86;
    }
};
__device__ __forceinline__ Mass to_mass(double w) {
    Mass m;
    const double h = w * 0x1p43;
    m.hi = (unsigned long long)h;
    m.lo = (unsigned long long)((h - (double)m.hi) * 0x1p43);
    return m;
}

struct Settings {
    float t, p, s;
    int k;
    bool bad;
};

// Settings of request i; k = 0: off, p = 1: off, s = 0: off.
__device__ __forceinline__ Settings settings(const sv_sampling& a, int i, int vocab) {
    Settings o;
    o.t = a.temperature != nullptr ? a.temperature[i] : 1.0f;
    o.k = a.top_k != nullptr ? a.top_k[i] : 0;
    o.p = a.top_p != nullptr ? a.top_p[i] : 1.0f;
    o.s = a.min_p != nullptr ? a.min_p[i] : 0.0f;
    o.bad = !(o.t >= 0.0f && o.t < kInf) || !(o.p >= 0.0f) || !(o.s >= 0.0f && o.s <= 1.0f);
    if (o.k <= 0 || o.k >= vocab) o.k = 0;
    if (o.p > 1.0f) o.p = 1.0f;
    return o;
}

// The ids of a law and their weights.
struct Weigher {
    double m, it;   // largest logit, 1 / T (0: T = 0, one id of weight 1)
    double s;       // min-p
    uint32_t ckey;  // the last logit's key and, among its ids, the last id
    int32_t cid;
    __device__ __forceinline__ bool above(uint32_t key, int id) const {
        return key > ckey || (key == ckey && id <= cid);
    }
    __device__ __forceinline__ double raw(float z) const { return exp(((double)z - m) * it); }
    __device__ __forceinline__ double operator()(float z, int id) const {
        if (!above(order_key(z), id)) return 0.0;
        const double w = raw(z);
        return w >= s ? w : 0.0;
    }
};

struct Smem {
    unsigned long long hi[256], lo[256];
    uint32_t cnt[256];
    uint32_t list_key[kList];
    int32_t list_id[kList];
    int list_n;
    uint32_t red[kWaves];
    int redi[kWaves];
    double redd[kWaves];
    // what a scan of the bins found
    uint32_t digit, before_cnt, in_cnt;
    int found;
    Mass before;
};

// One row, as granules of 8 ids.  Granule i starts at a 16-byte boundary and
// holds ids 8 i - shift .. + 7; the first and last may be partly outside.  Wave
// w holds the granules w * per .. + per - 1, in id order over (wave, step,
// lane).
template <sv_dtype DT>
struct Row {
    const char* base;  // the row's start, rounded down to 16 bytes
    int vocab, shift, per, steps;
    static constexpr int kBytes = DT == SV_BF16 ? 2 : 4;

    __device__ __forceinline__ Row(const char* row, int v) : vocab(v) {
        shift = (int)((reinterpret_cast<uintptr_t>(row) & 15) / kBytes);
        base = row - shift * kBytes;
        const int n = (v + shift + 7) / 8;
        per = ((n + kWaves - 1) / kWaves + kWave - 1) / kWave * kWave;
        steps = per / kWave;
    }
    __device__ __forceinline__ int first_id(int wave, int step, int lane) const {
        return (wave * per + step * kWave + lane) * 8 - shift;
    }
    // The 8 logits at ids id0 .. id0 + 7 (-inf outside the row).
    __device__ __forceinline__ void load(int id0, float* z) const {
        if (id0 >= 0 && id0 + 8 <= vocab) {
            const char* at = base + (int64_t)(id0 + shift) * kBytes;
            if (DT == SV_BF16) {
                const uint4 w = *reinterpret_cast<const uint4*>(at);
                z[0] = bf16_lo(w.x), z[1] = bf16_hi(w.x), z[2] = bf16_lo(w.y);
                z[3] = bf16_hi(w.y), z[4] = bf16_lo(w.z), z[5] = bf16_hi(w.z);
                z[6] = bf16_lo(w.w), z[7] = bf16_hi(w.w);
            } else {
                const float4 a = reinterpret_cast<const float4*>(at)[0];
                const float4 b = reinterpret_cast<const float4*>(at)[1];
                z[0] = a.x, z[1] = a.y, z[2] = a.z, z[3] = a.w;
                z[4] = b.x, z[5] = b.y, z[6] = b.z, z[7] = b.w;
            }
            return;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int id = id0 + e;
            z[e] = -kInf;
            if (id >= 0 && id < vocab) z[e] = one(id);
        }
    }
    __device__ __forceinline__ float one(int id) const {
        const char* at = base + (int64_t)(id + shift) * kBytes;
        if (DT == SV_BF16)
            return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(at) << 16);
        return *reinterpret_cast<const float*>(at);
    }
    // f(logit, id) over the calling thread's ids
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        for (int s = 0; s < steps; ++s) {
            const int id0 = first_id(wave, s, lane);
            if (id0 >= vocab) break;
            float z[8];
            load(id0, z);
#pragma unroll
            for (int e = 0; e < 8; ++e) f(z[e], id0 + e);
        }
    }
};

// ------------------------------------------------------- workgroup reductions

__device__ __forceinline__ uint32_t block_max(uint32_t v, Smem& sm) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
    __syncthreads();
    if (lane == 0) sm.red[wave] = v;
    __syncthreads();
    uint32_t r = sm.red[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) r = max(r, sm.red[w]);
    return r;
}

__device__ __forceinline__ int block_sum(int v, Smem& sm) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    v = wave_sum(v);
    __syncthreads();
    if (lane == 0) sm.redi[wave] = v;
    __syncthreads();
    int r = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) r += sm.redi[w];
    return r;
}

// Sums in a fixed order; also leaves each wave's own sum in sm.redd.
__device__ __forceinline__ double block_sum(double v, Smem& sm) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    v = wave_sum(v);
    __syncthreads();
    if (lane == 0) sm.redd[wave] = v;
    __syncthreads();
    double r = 0.0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) r += sm.redd[w];
    return r;
}

// ------------------------------------------------------------- digit descent

// Finds the first bin, in ascending order, whose running total reaches the
// target (count: >= want; mass: >= goal, or > goal if strict).  If none does,
// found = 0 and the bin is the last one that holds any mass.
template <bool MASS>
__device__ __forceinline__ void scan_bins(Smem& sm, uint32_t want, double goal, bool strict,
                                          Mass before, uint32_t before_cnt) {
    __syncthreads();
    if (threadIdx.x < kWave) {
        const int lane = threadIdx.x;
        unsigned long long h[4], l[4];
        uint32_t c[4];
        unsigned long long hs = 0, ls = 0;
        uint32_t cs = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] = sm.cnt[4 * lane + i];
            cs += c[i];
            if (MASS) {
                h[i] = sm.hi[4 * lane + i];
                l[i] = sm.lo[4 * lane + i];
                hs += h[i];
                ls += l[i];
            }
        }
        uint32_t cb = before_cnt + wave_incl_sum_dpp(cs, lane) - cs;
        Mass b = before;
        if (MASS) {
            b.hi += wave_incl_sum_dpp(hs, lane) - hs;
            b.lo += wave_incl_sum_dpp(ls, lane) - ls;
        }
        int at = -1, last = -1;
        Mass ab{0, 0}, lb{0, 0};
        uint32_t ac = 0, lc = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            bool hit;
            if (MASS) {
                const Mass n{b.hi + h[i], b.lo + l[i]};
                const double v = n.value();
                hit = c[i] != 0 && (strict ? v > goal : v >= goal);
            } else {
                hit = c[i] != 0 && cb + c[i] >= want;
            }
            if (hit && at < 0) at = i, ab = b, ac = cb;
            const bool any = MASS ? (h[i] | l[i]) != 0 : c[i] != 0;
            if (any) last = i, lb = b, lc = cb;
            cb += c[i];
            if (MASS) b.hi += h[i], b.lo += l[i];
        }
        const unsigned long long hits = __ballot(at >= 0), lasts = __ballot(last >= 0);
        const bool found = hits != 0;
        const int owner = found ? __builtin_ctzll(hits) : lasts ? 63 - __builtin_clzll(lasts) : 0;
        if (lane == owner) {
            const int i = found ? at : last < 0 ? 0 : last;
            sm.digit = 4 * lane + i;
            sm.before = found ? ab : lb;
            sm.before_cnt = found ? ac : lc;
            sm.in_cnt = sm.cnt[4 * lane + i];
            sm.found = found;
        }
    }
    __syncthreads();
}

struct Found {
    uint32_t ord;         // the ordinal (low bits below the last digit 0)
    uint32_t before_cnt;  // what takes part ahead of it
    uint32_t in_cnt;      // what has it
    Mass before;
    bool found;
};

// The border among the ordinals of what takes part: each(f) calls f(ord) or,
// with masses, f(ord, w) for every part-taker of the calling thread.
template <bool MASS, class Each>
__device__ Found descend(Smem& sm, Each each, int top, int low, uint32_t want, double goal,
                         bool strict) {
    Found r{0, 0, 0, {0, 0}, true};
    for (int sh = top; sh >= low; sh -= 8) {
        __syncthreads();
        for (int i = threadIdx.x; i < 256; i += blockDim.x) {
            sm.cnt[i] = 0;
            if (MASS) sm.hi[i] = sm.lo[i] = 0;
        }
        __syncthreads();
        const uint32_t prefix = r.ord;
        each([&](uint32_t ord, auto weight) {
            if (((uint64_t)(ord ^ prefix) >> (sh + 8)) != 0) return;
            const int i = (ord >> sh) & 255;
            atomicAdd(&sm.cnt[i], 1u);
            if (MASS) {
                const Mass m = to_mass(weight());
                if (m.hi) atomicAdd(&sm.hi[i], m.hi);
                if (m.lo) atomicAdd(&sm.lo[i], m.lo);
            }
        });
        // once a level found no border, the search goes for the last mass
        scan_bins<MASS>(sm, want, r.found ? goal : (double)kInf, strict, r.before, r.before_cnt);
        r.ord |= sm.digit << sh;
        r.before_cnt = sm.before_cnt;
        r.in_cnt = sm.in_cnt;
        r.before = sm.before;
        r.found = r.found && sm.found;
    }
    return r;
}

// --------------------------------------------------------------- the law

struct Result {
    Weigher w;
    int n;         // ids in the support
    double total;  // their weight
    bool listed;   // the candidates are in sm.list_*
    int fault;     // SV_DEV_* bits
};

// Calls f(logit, id) for the candidates of the calling thread.
template <sv_dtype DT, class F>
__device__ __forceinline__ void candidates(const Row<DT>& row, const Smem& sm, bool listed, F f) {
    if (listed) {
        for (int i = threadIdx.x; i < sm.list_n; i += kThreads)
            f(key_logit(sm.list_key[i]), sm.list_id[i]);
    } else {
        row.each(f);
    }
}

// Low bit of the key digits that differ between logits: a bf16's lower half
// is the same for all of one sign.
template <sv_dtype DT>
constexpr int kLowDigit = DT == SV_BF16 ? 16 : 0;

// A descent's ordinal is the complement of the key: larger logits first.
template <sv_dtype DT>
__device__ __forceinline__ uint32_t ordinal_key(uint32_t ord) {
    uint32_t key = ~ord;
    if (DT == SV_BF16) key = (key & 0xffff0000u) | ((key >> 31) ? 0u : 0xffffu);
    return key;
}

template <sv_dtype DT>
__device__ Result find_law(const Row<DT>& row, const Settings& set, Smem& sm) {
    Result r{};
    // pass 1: largest logit, faults
    uint32_t mine = 0;
    int bad = 0;
    row.each([&](float z, int id) {
        mine = max(mine, order_key(z));
        bad |= !(z < kInf);  // NaN or +inf
    });
    const uint32_t top = block_max(mine, sm);
    bad = __syncthreads_or(bad);
    if (bad || top <= kMinusInfKey) r.fault |= SV_DEV_NONFINITE;
    if (set.bad) r.fault |= SV_DEV_BAD_PARAM;
    if (r.fault) return r;
    const float m = key_logit(top);
    Weigher& w = r.w;
    w.m = (double)m;
    w.s = 0.0;
    w.ckey = kMinusInfKey;
    w.cid = INT32_MIN;  // ids of -inf (and those before the row, read as -inf) never count

    if (set.t == 0.0f) {
        // the lowest id of the largest logit
        uint32_t first = 0;
        row.each([&](float z, int id) {
            if (order_key(z) == top) first = max(first, ~(uint32_t)id);
        });
        w.it = 0.0;
        w.ckey = top;
        w.cid = (int)~block_max(first, sm);
        r.n = 1;
        r.total = 1.0;
        return r;
    }
    w.it = 1.0 / (double)set.t;

    // lb: no id below this logit is in the support (nor, with top-k, among
    // the first k)
    const bool use_p = set.p < 1.0f;
    float lb = -kInf;
    if (set.k > 0 && set.k <= kThreads) {
        // the k-th largest of the threads' maxima: k ids are at least that
        const Found f = descend<false>(
            sm, [&](auto fn) { if (mine > kMinusInfKey) fn(~mine, [] { return 0.0; }); }, 24,
            kLowDigit<DT>, (uint32_t)set.k, 0.0, false);
        if (f.found) lb = key_logit(ordinal_key<DT>(f.ord));
    }
    if (set.s > 0.0f && !(use_p && set.k > 0)) {
        // a little below m + T ln s, for the roundings on the way (of the
        // logits' size, and of an exponent's: weights next to 1 round to 1)
        const double z = w.m + log((double)set.s) / w.it;
        const double slack = 1e-6 * (fabs(w.m) + fabs(z) + (double)set.t);
        lb = fmaxf(lb, (float)(z - slack));
    }
    double total = 0.0;
    if (use_p && set.k == 0) {
        double part = 0.0;
        row.each([&](float z, int id) { if (z > -kInf) part += w.raw(z); });
        total = block_sum(part, sm);
        // all ids below lb together weigh less than what top-p leaves out
        const double left = (1.0 - (double)set.p) * total / (double)row.vocab;
        const double z = w.m + log(left) / w.it;
        const double slack = 1e-6 * (fabs(w.m) + fabs(z) + (double)set.t);
        lb = fmaxf(lb, (float)(z - slack));
    }
    // keep what is left in LDS if it fits
    r.listed = lb > -kInf;
    if (r.listed) {
        if (threadIdx.x == 0) sm.list_n = 0;
        __syncthreads();
        row.each([&](float z, int id) {
            if (z >= lb) {
                const int at = atomicAdd(&sm.list_n, 1);
                if (at < kList) {
                    sm.list_key[at] = order_key(z);
                    sm.list_id[at] = id;
                }
            }
        });
        __syncthreads();
        r.listed = sm.list_n <= kList;
    }
    const auto in = [&](float z) { return z >= lb && z > -kInf; };

    // a border after `want` of the ids at key ckey, of which in_cnt take part
    const auto cut_ties = [&](uint32_t key, uint32_t want, uint32_t in_cnt) {
        int cid = INT32_MAX;
        if (want < in_cnt) {
            const Weigher was = w;
            const Found f = descend<false>(
                sm,
                [&](auto fn) {
                    candidates(row, sm, r.listed, [&](float z, int id) {
                        if (order_key(z) == key && was.above(key, id))
                            fn((uint32_t)id, [] { return 0.0; });
                    });
                },
                16, 0, want, 0.0, false);
            cid = (int)f.ord;
        }
        w.ckey = key;
        w.cid = cid;
    };

    if (set.k > 0) {
        const Found f = descend<false>(
            sm,
            [&](auto fn) {
                candidates(row, sm, r.listed, [&](float z, int id) {
                    if (in(z)) fn(~order_key(z), [] { return 0.0; });
                });
            },
            24, kLowDigit<DT>, (uint32_t)set.k, 0.0, false);
        if (f.found)
            cut_ties(ordinal_key<DT>(f.ord), (uint32_t)set.k - f.before_cnt, f.in_cnt);
    }
    if (use_p) {
        if (set.k > 0) {
            double part = 0.0;
            if (r.listed) {
                // the list's order is not fixed: gathered in fixed point
                __syncthreads();
                if (threadIdx.x == 0) sm.hi[0] = sm.lo[0] = 0;
                __syncthreads();
                candidates(row, sm, true, [&](float z, int id) {
                    if (w.above(order_key(z), id)) {
                        const Mass x = to_mass(w.raw(z));
                        atomicAdd(&sm.hi[0], x.hi);
                        atomicAdd(&sm.lo[0], x.lo);
                    }
                });
                __syncthreads();
                total = Mass{sm.hi[0], sm.lo[0]}.value();
            } else {
                row.each([&](float z, int id) {
                    if (w.above(order_key(z), id)) part += w.raw(z);
                });
                total = block_sum(part, sm);
            }
        }
        const double goal = (double)set.p * total;
        const Found f = descend<true>(
            sm,
            [&](auto fn) {
                candidates(row, sm, r.listed, [&](float z, int id) {
                    if (in(z) && w.above(order_key(z), id))
                        fn(~order_key(z), [&] { return w.raw(z); });
                });
            },
            24, kLowDigit<DT>, 0, goal, false);
        if (f.found) {
            const uint32_t key = ordinal_key<DT>(f.ord);
            const double one = w.raw(key_logit(key));
            double want = one > 0.0 ? ceil((goal - f.before.value()) / one) : 1.0;
            want = fmin(fmax(want, 1.0), (double)f.in_cnt);
            cut_ties(key, (uint32_t)want, f.in_cnt);
        }
    }
    w.s = (double)set.s;

    // how many, and their weight
    int n = 0;
    if (r.listed) {
        __syncthreads();
        if (threadIdx.x == 0) sm.hi[0] = sm.lo[0] = 0;
        __syncthreads();
        candidates(row, sm, true, [&](float z, int id) {
            if (!w.above(order_key(z), id)) return;
            const double x = w.raw(z);
            if (x < w.s) return;
            ++n;
            const Mass q = to_mass(x);
            atomicAdd(&sm.hi[0], q.hi);
            atomicAdd(&sm.lo[0], q.lo);
        });
        r.n = block_sum(n, sm);
        r.total = Mass{sm.hi[0], sm.lo[0]}.value();
        __syncthreads();
    } else {
        double part = 0.0;
        row.each([&](float z, int id) {
            if (!w.above(order_key(z), id)) return;
            const double x = w.raw(z);
            if (x < w.s) return;
            ++n;
            part += x;
        });
        r.n = block_sum(n, sm);
        r.total = block_sum(part, sm);  // leaves the waves' sums in sm.redd
    }
    return r;
}

// The smallest id whose running sum, over a row in wave segments, passes goal:
// the waves' sums are in sm.redd; the wave that holds the crossing walks its
// segment again.  sum8(id0, x) gives the 8 weights at ids id0 .. id0 + 7.
// If rounding leaves none, the last id of positive weight.
template <class Sum8, class FirstId>
__device__ int walk_row(Smem& sm, double goal, int steps, FirstId first_id, int vocab, Sum8 sum8) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    double before = 0.0;
    int owner = -1;
    for (int w = 0; w < kWaves; ++w) {
        if (before + sm.redd[w] > goal) {
            owner = w;
            break;
        }
        before += sm.redd[w];
    }
    if (owner < 0) {
        goal = kInf;
        before = 0.0;
        for (int w = 0; w < kWaves; ++w)
            if (sm.redd[w] > 0.0) owner = w;
    }
    if (wave == owner) {
        int tok = -1, last = -1;
        for (int s = 0; s < steps && tok < 0; ++s) {
            const int id0 = first_id(owner, s, lane);
            double x[8], mine = 0.0;
            if (id0 < vocab) {
                sum8(id0, x);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = 0.0;
            }
            int mylast = -1;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                mine += x[e];
                if (x[e] > 0.0) mylast = id0 + e;
            }
            const double incl = wave_incl_sum_dpp(mine, lane);
            double c = before + (incl - mine);
            int hit = -1;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                c += x[e];
                if (hit < 0 && x[e] > 0.0 && c > goal) hit = id0 + e;
            }
            const unsigned long long hits = __ballot(hit >= 0), some = __ballot(mylast >= 0);
            if (hits) tok = __builtin_amdgcn_readlane(hit, __builtin_ctzll(hits));
            if (some) last = __builtin_amdgcn_readlane(mylast, 63 - __builtin_clzll(some));
            before += lane63(incl);
        }
        if (lane == 0) sm.redi[0] = tok >= 0 ? tok : last;
    }
    __syncthreads();
    return sm.redi[0];
}

// The id a uniform u in [0, 1) draws from a law find_law has just made.
template <sv_dtype DT>
__device__ int draw(const Row<DT>& row, const Result& r, float u, Smem& sm) {
    if (r.w.it == 0.0) return r.w.cid;
    const double goal = (double)u * r.total;
    if (!r.listed) {
        return walk_row(
            sm, goal, row.steps,
            [&](int w, int s, int l) { return row.first_id(w, s, l); }, row.vocab,
            [&](int id0, double* x) {
                float z[8];
                row.load(id0, z);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = r.w(z[e], id0 + e);
            });
    }
    const auto live = [&](auto fn) {
        candidates(row, sm, true, [&](float z, int id) {
            const double x = r.w(z, id);
            if (x > 0.0) fn((uint32_t)id, [&] { return x; });
        });
    };
    // u = 0: the lowest id of any weight, however small
    if (u == 0.0f) return (int)descend<false>(sm, live, 16, 0, 1, 0.0, false).ord;
    return (int)descend<true>(sm, live, 16, 0, 0, goal, true).ord;
}

}  // namespace law
}  // namespace sv
