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
// One workgroup takes a row.  Four ways to the border, by what the settings ask
// for (times: calls of 256 rows, one a workgroup, normal logits of spread 3, T =
// 1; the pass over memory that finds the largest logit and the faults is part of
// each):
//  - T = 0, top-k up to the workgroup's threads, or min-p: a bound that costs no
//    pass (the largest logit, the k-th largest of the threads' own maxima,
//    min-p's logit) leaves a few candidates, which are gathered in LDS, ranked by
//    counting and summed there (T = 0, top-k of 50, min-p of 0.05: 129,280 bf16
//    17, 24, 34 us; 256,000 fp32 44, 54, 67).  Near the thread count top-k leaves
//    more of them than the list holds (of 1024 threads: 50 us at 512, 131 at 1024);
//  - bf16, top-p alone, and no cut where no draw follows: how many ids have each
//    value, counted in the first pass, gives the sum and the border (by_value();
//    53 us with a draw; 67 at T = 2, 98 at T = 5, where more than 256 ids lie below
//    the 16 octaves of values and are counted over);
//  - fp32, top-p alone, and no cut: the first pass takes the sum, and top-p's
//    histogram over 2048 steps of the weight (2^(1/32) each); the steps next to
//    the border are gathered and searched like candidates while the ids above
//    them are summed (find_nucleus(); 134 us, 69 without top-p);
//  - anything else, and what does not fit the lists (long runs of equal logits,
//    fp32 top-p with thousands of ids in the border's step, 807 us at T = 2):
//    the border is found digit by digit, 256 bins over 8 bits of the ordered key,
//    then the next 8 bits within the bin that holds the border (top-k of 2000 of
//    129,280 bf16: 128 us).
#pragma once

#include "sv_device.h"
#include "sv_serve.h"

namespace sv {
namespace law {

constexpr int kCUs = 256;    // of an MI355X
constexpr int kList = 2048;  // candidates kept in LDS
constexpr int kRank = 256;   // candidates ranked by counting
constexpr int kSteps = 2048; // histogram of the weights, kPerOctave steps for a factor of 2
constexpr float kPerOctave = 32.0f;
constexpr int kAbove = 640;  // of them above the logit they start from
constexpr double kLog2e64 = 1.4426950408889634074;
constexpr int kValues = 2048;  // bf16 values of either sign counted by value: 16 octaves
constexpr int kQueue = 640;  // ids a wave keeps for compact(): 64 left over and 512 of a step
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

// 2^t for t <= 0, to 4e-14: t = n + r with n an integer and |r| <= 1/2, 2^r = 1 +
// r q(r) with q of degree 8 through the Chebyshev nodes of [-1/2, 1/2].  2^0 is
// exactly 1, so equal logits have equal weights, and counts of them are exact.
// Some eighteen fp64 operations an id (4.1 clocks a wave each) bound the passes
// that sum a row: 18 us for 129,280 ids on one CU.
__device__ __forceinline__ double pow2(double t) {
    t = fmax(t, -1100.0);
    const double shifted = t + 0x1.8p52;
    const int n = (int)(uint32_t)(uint64_t)__double_as_longlong(shifted);
    const double r = t - (shifted - 0x1.8p52);
    double q = 0x1.b63880a30e9ffp-24;
    q = fma(q, r, 0x1.63d136366db24p-20);
    q = fma(q, r, 0x1.ffcb9515a8016p-17);
    q = fma(q, r, 0x1.4308ac85aa947p-13);
    q = fma(q, r, 0x1.5d87fe86fe88ep-10);
    q = fma(q, r, 0x1.3b2ab7181b755p-7);
    q = fma(q, r, 0x1.c6b08d7047e52p-5);
    q = fma(q, r, 0x1.ebfbdff823cedp-3);
    q = fma(q, r, 0x1.62e42fefa39efp-1);
    return __builtin_amdgcn_ldexp(fma(q, r, 1.0), n);
}

// The ids of a law and their weights: logits above zc, and those equal to it
// up to id cid, of weight at least s.
struct Weigher {
    double m, it;  // largest logit, log2(e) / T (0: T = 0, one id of weight 1)
    double s;      // min-p
    float zc;
    int32_t cid;
    __device__ __forceinline__ bool above(float z, int id) const {
        return z > zc || (z == zc && id <= cid);
    }
    __device__ __forceinline__ double raw(float z) const { return pow2(((double)z - m) * it); }
    __device__ __forceinline__ double operator()(float z, int id) const {
        const double w = raw(z);
        return above(z, id) && w >= s ? w : 0.0;
    }
};

template <int NT>
struct Smem {
    static constexpr int kWaves = NT / kWave;
    static constexpr int kBatches = 8192 / NT;
    static constexpr int kMaxSteps = (SV_MAX_VOCAB + 8) / 8 / NT + 1;  // of a wave's segment
    uint32_t step[kSteps];             // histogram of the weights
    unsigned long long list[kList];    // candidates: key, then ~id: larger is earlier
    unsigned long long sorted[kRank];  // ranked
    double weight[kRank];
    double prefix[kRank];
    double seg[kMaxSteps];
    union {
        struct {  // compact()
            float queue_z[kWaves][kQueue];
            int queue_id[kWaves][kQueue];
        };
        uint32_t value[2 * kValues + kWave];  // by_value(): how many ids have each logit
        uint16_t batch_top[kBatches][NT];  // pass 1: key of each batch's largest logit
    };
    unsigned long long hi[256], lo[256];
    uint32_t cnt[256];
    int list_n;
    uint32_t red[NT / kWave];
    int redi[NT / kWave];
    double redd[NT / kWave];
    int first, second;
    // what a scan of the bins found
    uint32_t digit, before_cnt, in_cnt;
    int found;
    Mass before;
};

__device__ __forceinline__ unsigned long long entry(uint32_t key, int id) {
    return ((unsigned long long)key << 32) | (uint32_t)~id;
}
__device__ __forceinline__ uint32_t entry_key(unsigned long long e) { return (uint32_t)(e >> 32); }
__device__ __forceinline__ int entry_id(unsigned long long e) { return (int)~(uint32_t)e; }

// One row, as granules of 8 ids (8 i .. 8 i + 7).  Wave w holds the granules w *
// per .. + per - 1, in id order over (wave, step, lane).  Loads are 16 bytes
// wherever a row starts: the hardware takes them at any element.
template <sv_dtype DT, int NT>
struct Row {
    static constexpr int kWaves = NT / kWave;
    const char* base;
    int vocab, per, steps;
    static constexpr int kBytes = DT == SV_BF16 ? 2 : 4;
    static constexpr int kWords = 2 * kBytes;
    static constexpr uint32_t kFill = DT == SV_BF16 ? 0xff80ff80u : 0xff800000u;  // -inf

    // segments: one for each of the workgroup's waves, or more
    __device__ __forceinline__ Row(const char* row, int v, int segments = kWaves)
        : base(row), vocab(v) {
        const int n = (v + 7) / 8;
        per = ((n + segments - 1) / segments + kWave - 1) / kWave * kWave;
        steps = per / kWave;
    }
    __device__ __forceinline__ int first_id(int wave, int step, int lane) const {
        return (wave * per + step * kWave + lane) * 8;
    }
    // 8 logits as they lie in memory
    struct Raw {
        uint32_t w[2 * kBytes];
        __device__ __forceinline__ void unpack(float* z) const {
            if (DT == SV_BF16) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    z[2 * i] = bf16_lo(w[i]);
                    z[2 * i + 1] = bf16_hi(w[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] = __uint_as_float(w[i % (2 * kBytes)]);
            }
        }
    };
    // 16-byte loads of the granule at id0; the row's last granule as its last 8
    // ids, which settle() moves down.  A launch of one wave a row is for rows
    // of fewer than 8 ids, read one by one.
    __device__ __forceinline__ Raw fetch(int id0) const {
        Raw out;
        if constexpr (NT == kWave) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) out.w[i] = kFill;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (id0 != 0 || e >= vocab) break;
                const uint32_t z = __float_as_uint(one(e));
                if (DT == SV_F32) out.w[e % kWords] = z;
                else if (e & 1) out.w[e / 2] = (out.w[e / 2] & 0xffffu) | z;
                else out.w[e / 2] = (out.w[e / 2] & 0xffff0000u) | (z >> 16);
            }
        } else {
            __builtin_memcpy(out.w, base + (int64_t)min(id0, vocab - 8) * kBytes, sizeof(out.w));
        }
        return out;
    }
    // Ids past the row's end read as -inf.
    __device__ __forceinline__ void settle(Raw& g, int id0) const {
        if constexpr (NT == kWave) return;
        const int over = id0 + 8 - vocab;
        if (over <= 0) return;
        int by_words = over;
        if (DT == SV_BF16) {
            if (over & 1) {
#pragma unroll
                for (int i = 0; i < kWords; ++i)
                    g.w[i] = (g.w[i] >> 16) |
                             (i + 1 < kWords ? g.w[(i + 1) % kWords] << 16 : 0xff800000u);
            }
            by_words = over >> 1;
        }
#pragma unroll
        for (int by = 1; by < kWords; by *= 2) {
            if (by_words & by) {
#pragma unroll
                for (int i = 0; i < kWords; ++i)
                    g.w[i] = i + by < kWords ? g.w[(i + by) % kWords] : kFill;
            }
        }
        if (over >= 8) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) g.w[i] = kFill;
        }
    }
    __device__ __forceinline__ Raw raw(int id0) const {
        Raw g = fetch(id0);
        settle(g, id0);
        return g;
    }
    // Whether a step of the wave holds ids past the row's end (the same in
    // every lane).
    __device__ __forceinline__ bool ends_in(int wave, int step) const {
        return __builtin_amdgcn_readfirstlane(first_id(wave, step, kWave - 1)) + 8 > vocab;
    }
    __device__ __forceinline__ void load(int id0, float* z) const { raw(id0).unpack(z); }
    __device__ __forceinline__ float one(int id) const {
        const char* at = base + (int64_t)id * kBytes;
        if (DT == SV_BF16)
            return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(at) << 16);
        return *reinterpret_cast<const float*>(at);
    }
    // The wave that holds an id.
    __device__ __forceinline__ int wave_of(int id) const { return (id >> 3) / per; }
    // The same granules dealt to the threads in turn, for passes whose order
    // does not matter.
    __device__ __forceinline__ int turn_id(int s) const {
        return (s * NT + (int)threadIdx.x) * 8;
    }
    __device__ __forceinline__ int turns() const { return (vocab + 8 * NT - 1) / (8 * NT); }
    // f(granule, first id) over the granules dealt to the calling thread, kAhead
    // loads of them at a time, done(batch) after each.  Granules outside the row
    // read as -inf.
    template <int kAhead, class F, class Done>
    __device__ __forceinline__ void granules(F f, Done done) const {
        const int n = turns();
        int s = 0;
        for (; (s + kAhead) * NT * 8 <= vocab; s += kAhead) {
            Raw g[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) g[i] = fetch(turn_id(s + i));
#pragma unroll
            for (int i = 0; i < kAhead; ++i) f(g[i], turn_id(s + i));
            done(s / kAhead);
        }
        if (s >= n) return;
        // the last batch, its loads in flight together too (taken one by one
        // they cost a pass over 129,280 ids a third of its time)
        const int end = vocab & ~7;
        Raw g[kAhead], part = fetch(end);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) g[i] = fetch(turn_id(s + i));
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (turn_id(s + i) < end) f(g[i], turn_id(s + i));
        if (end < vocab && (int)threadIdx.x == end / 8 % NT) {
            settle(part, end);
            f(part, end);
        }
        done(s / kAhead);
    }
    // f(granule, first id), one granule at a time, the next one in flight; lanes
    // whose granule is outside the row take part with logits of -inf
    template <class F>
    __device__ __forceinline__ void granules_of(int wave, int lane, F f) const {
        int id0 = first_id(wave, 0, lane);
        Raw next = fetch(id0);
        for (int s = 0; s < steps; ++s) {
            if (first_id(wave, s, 0) >= vocab) break;
            Raw now = next;
            const int id1 = first_id(wave, s + 1, lane);
            if (s + 1 < steps) next = fetch(id1);
            if (ends_in(wave, s)) settle(now, id0);
            f(now, id0);
            id0 = id1;
        }
    }
    // f(granule, first id) over the calling wave's granules in id order, kAhead
    // loads of them at a time
    template <int kAhead, class F>
    __device__ __forceinline__ void in_order(F f) const {
        in_order<kAhead>(threadIdx.x >> 6, f);
    }
    template <int kAhead, class F>
    __device__ __forceinline__ void in_order(int wave, F f) const {
        const int lane = threadIdx.x & 63;
        for (int s = 0; s < steps && first_id(wave, s, 0) < vocab; s += kAhead) {
            Raw g[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) g[i] = fetch(first_id(wave, s + i, lane));
            if (ends_in(wave, s + kAhead - 1)) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) settle(g[i], first_id(wave, s + i, lane));
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (s + i < steps) f(g[i], first_id(wave, s + i, lane));
        }
    }
    template <class F>
    __device__ __forceinline__ void each_granule(F f) const {
        granules_of(threadIdx.x >> 6, threadIdx.x & 63, f);
    }
    // f(logit, id) over the calling thread's ids
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        each_granule([&](const Raw& g, int id0) {
            float z[8];
            g.unpack(z);
#pragma unroll
            for (int e = 0; e < 8; ++e) f(z[e], id0 + e);
        });
    }
};

// Calls use(logit, id) for the ids that keep(logit) leaves, 64 of a wave at a
// time and in id order within the wave, the last call with fewer lanes.  Where
// a few per cent of the ids are kept, the work on them then costs a wave per 64
// of them and not nearly a wave per 64 ids of the row (129,280 ids, 2 % kept:
// 30 us for the sum of their weights id by id, 9 this way).  kAhead: loads in
// flight together, 1: the next one while one is worked on.
template <int kAhead = 1, sv_dtype DT, int NT, class Keep, class Use>
__device__ __forceinline__ void compact(const Row<DT, NT>& row, Smem<NT>& sm, int segment, Keep keep,
                                        Use use) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float* qz = sm.queue_z[wave];
    int* qi = sm.queue_id[wave];
    int n = 0;  // the same in every lane
    const auto take = [&](const typename Row<DT, NT>::Raw& g, int id0) {
        float z[8];
        g.unpack(z);
        int c = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) c += keep(z[e]) ? 1 : 0;
        if (__ballot(c != 0) == 0) return;
        const int incl = wave_incl_sum_dpp(c, lane);
        int at = n + incl - c;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (keep(z[e])) {
                qz[at] = z[e];
                qi[at] = id0 + e;
                ++at;
            }
        }
        n += lane63(incl);
        __builtin_amdgcn_wave_barrier();
        int head = 0;
        for (; n - head >= kWave; head += kWave) use(qz[head + lane], qi[head + lane]);
        if (head > 0) {
            n -= head;
            float mz = 0.0f;
            int mi = 0;
            if (lane < n) mz = qz[head + lane], mi = qi[head + lane];
            __builtin_amdgcn_wave_barrier();
            if (lane < n) qz[lane] = mz, qi[lane] = mi;
            __builtin_amdgcn_wave_barrier();
        }
    };
    if constexpr (kAhead > 1) row.template in_order<kAhead>(segment, take);
    else row.granules_of(segment, lane, take);
    if (lane < n) use(qz[lane], qi[lane]);
}

// Largest logit and faults of a thread's ids, on the raw words: positive floats
// order as signed integers, negative ones backwards as unsigned.
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
template <sv_dtype DT>
struct Extremes;
template <>
struct Extremes<SV_BF16> {
    s16x2 smax{-32768, -32768};
    u16x2 umax{0, 0}, umin{0xffff, 0xffff};
    __device__ __forceinline__ void add(uint32_t w) {
        smax = __builtin_elementwise_max(smax, __builtin_bit_cast(s16x2, w));
        umax = __builtin_elementwise_max(umax, __builtin_bit_cast(u16x2, w));
        umin = __builtin_elementwise_min(umin, __builtin_bit_cast(u16x2, w));
    }
    __device__ __forceinline__ void add(const Extremes& o) {
        smax = __builtin_elementwise_max(smax, o.smax);
        umax = __builtin_elementwise_max(umax, o.umax);
        umin = __builtin_elementwise_min(umin, o.umin);
    }
    __device__ __forceinline__ uint32_t top() const {
        const int s = max(smax.x, smax.y);
        const uint32_t b = s >= 0 ? (uint32_t)s : (uint32_t)min(umin.x, umin.y);
        return order_key(__uint_as_float(b << 16));
    }
    __device__ __forceinline__ bool bad() const {  // NaN or +inf
        return max(smax.x, smax.y) >= 0x7f80 || max(umax.x, umax.y) > 0xff80;
    }
};
template <>
struct Extremes<SV_F32> {
    int32_t smax = INT32_MIN;
    uint32_t umax = 0, umin = 0xffffffffu;
    __device__ __forceinline__ void add(uint32_t w) {
        smax = max(smax, (int32_t)w);
        umax = max(umax, w);
        umin = min(umin, w);
    }
    __device__ __forceinline__ void add(const Extremes& o) {
        smax = max(smax, o.smax);
        umax = max(umax, o.umax);
        umin = min(umin, o.umin);
    }
    __device__ __forceinline__ uint32_t top() const {
        return order_key(__uint_as_float(smax >= 0 ? (uint32_t)smax : umin));
    }
    __device__ __forceinline__ bool bad() const {
        return smax >= 0x7f800000 || umax > 0xff800000u;
    }
};

// ------------------------------------------------------- workgroup reductions

template <int NT>
__device__ __forceinline__ uint32_t block_max(uint32_t v, Smem<NT>& sm) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
    __syncthreads();
    if (lane == 0) sm.red[wave] = v;
    __syncthreads();
    uint32_t r = sm.red[0];
#pragma unroll
    for (int w = 1; w < NT / kWave; ++w) r = max(r, sm.red[w]);
    return r;
}

template <int NT>
__device__ __forceinline__ int block_sum(int v, Smem<NT>& sm) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    v = wave_sum(v);
    __syncthreads();
    if (lane == 0) sm.redi[wave] = v;
    __syncthreads();
    int r = 0;
#pragma unroll
    for (int w = 0; w < NT / kWave; ++w) r += sm.redi[w];
    return r;
}

// Sums in a fixed order; also leaves each wave's own sum in sm.redd.
template <int NT>
__device__ __forceinline__ double block_sum(double v, Smem<NT>& sm) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    v = wave_sum(v);
    __syncthreads();
    if (lane == 0) sm.redd[wave] = v;
    __syncthreads();
    double r = 0.0;
#pragma unroll
    for (int w = 0; w < NT / kWave; ++w) r += sm.redd[w];
    return r;
}

// ------------------------------------------------------------- digit descent

// Finds the first bin, in ascending order, whose running total reaches the
// target (count: >= want; mass: >= goal, or > goal if strict).  If none does,
// found = 0 and the bin is the last one that holds any mass.
template <bool MASS, int NT>
__device__ __forceinline__ void scan_bins(Smem<NT>& sm, uint32_t want, double goal, bool strict,
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
        // of this lane's bins: the one found, and the last that holds any
        int at = -1, last = -1;
        unsigned long long at_hi = 0, at_lo = 0, last_hi = 0, last_lo = 0;
        uint32_t at_cnt = 0, last_cnt = 0;
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
            if (hit && at < 0) {
                at = i;
                at_hi = b.hi;
                at_lo = b.lo;
                at_cnt = cb;
            }
            const bool any = MASS ? (h[i] | l[i]) != 0 : c[i] != 0;
            if (any) {
                last = i;
                last_hi = b.hi;
                last_lo = b.lo;
                last_cnt = cb;
            }
            cb += c[i];
            if (MASS) {
                b.hi += h[i];
                b.lo += l[i];
            }
        }
        const unsigned long long hits = __ballot(at >= 0), lasts = __ballot(last >= 0);
        const bool found = hits != 0;
        const int owner = found ? __builtin_ctzll(hits) : lasts ? 63 - __builtin_clzll(lasts) : 0;
        if (lane == owner) {
            const int i = found ? at : last < 0 ? 0 : last;
            sm.digit = 4 * lane + i;
            sm.before.hi = found ? at_hi : last_hi;
            sm.before.lo = found ? at_lo : last_lo;
            sm.before_cnt = found ? at_cnt : last_cnt;
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
template <bool MASS, int NT, class Each>
__device__ Found descend(Smem<NT>& sm, Each each, int top, int low, uint32_t want, double goal,
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
        scan_bins<MASS, NT>(sm, want, r.found ? goal : (double)kInf, strict, r.before, r.before_cnt);
        r.ord |= sm.digit << sh;
        r.before_cnt = sm.before_cnt;
        r.in_cnt = sm.in_cnt;
        r.before = sm.before;
        r.found = r.found && sm.found;
    }
    return r;
}

// --------------------------------------------------------------- the law

// Where a law's ids are found again: ranked in sm.sorted (the first n), among
// sm.list, or in the row (with the waves' sums in sm.redd).
enum Where { kRanked, kListed, kInRow };

struct Result {
    Weigher w;
    int n;         // ids in the support
    double total;  // their weight
    Where where;
    int fault;     // SV_DEV_* bits
};

// Calls f(logit, id) for the candidates of the calling thread.
template <sv_dtype DT, int NT, class F>
__device__ __forceinline__ void candidates(const Row<DT, NT>& row, const Smem<NT>& sm, bool listed, F f) {
    if (listed) {
        for (int i = threadIdx.x; i < sm.list_n; i += NT)
            f(key_logit(entry_key(sm.list[i])), entry_id(sm.list[i]));
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

// Ranks sm.list (n <= kRank entries) into sm.sorted, with weights and running
// sums in that order.  The list's own order, which atomics made, does not show.
template <int NT>
__device__ __forceinline__ void rank_list(const Weigher& w, Smem<NT>& sm, int n) {
    const int i = threadIdx.x, lane = i & 63, wave = i >> 6;
    if (i < n) {
        const unsigned long long mine = sm.list[i];
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) rank += sm.list[j] > mine;
        sm.sorted[rank] = mine;
    }
    __syncthreads();
    double x = 0.0;
    if (i < n) x = w.raw(key_logit(entry_key(sm.sorted[i])));
    double incl = 0.0;
    if (wave < kRank / kWave) {
        incl = wave_incl_sum_dpp(x, lane);
        if (lane == 63) sm.redd[wave] = incl;
    }
    __syncthreads();
    if (i < n) {
        double before = 0.0;
        for (int v = 0; v < wave; ++v) before += sm.redd[v];
        sm.weight[i] = x;
        sm.prefix[i] = before + incl;
    }
    __syncthreads();
}

// The smallest i < n for which test(i) holds, else n (n <= NT).
template <int NT, class Test>
__device__ __forceinline__ int first_of(Smem<NT>& sm, int n, Test test) {
    const int i = threadIdx.x;
    const unsigned long long hits = __ballot(i < n && test(i));
    __syncthreads();
    if ((i & 63) == 0) sm.redi[i >> 6] = hits ? i + __builtin_ctzll(hits) : n;
    __syncthreads();
    int r = n;
#pragma unroll
    for (int w = 0; w < NT / kWave; ++w) r = min(r, sm.redi[w]);
    return r;
}

// Sums 64-bit weights of the listed ids that live(z, id) leaves, and counts
// them, whatever the list's order.
template <int NT, class Live>
__device__ __forceinline__ double sum_list(Smem<NT>& sm, const Weigher& w, int& n, Live live) {
    __syncthreads();
    if (threadIdx.x == 0) sm.hi[0] = sm.lo[0] = 0, sm.second = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < sm.list_n; i += NT) {
        const float z = key_logit(entry_key(sm.list[i]));
        const double x = w.raw(z);
        if (!live(z, entry_id(sm.list[i]), x)) continue;
        const Mass q = to_mass(x);
        atomicAdd(&sm.hi[0], q.hi);
        atomicAdd(&sm.lo[0], q.lo);
        atomicAdd(&sm.second, 1);
    }
    __syncthreads();
    n = sm.second;
    return Mass{sm.hi[0], sm.lo[0]}.value();
}

// Moves the border of w behind the first `want` of the ids (candidates that w
// has now) whose logit has this key, of which in_cnt take part.
template <sv_dtype DT, int NT>
__device__ __forceinline__ void cut_ties(const Row<DT, NT>& row, Smem<NT>& sm, bool listed, Weigher& w,
                                         uint32_t key, uint32_t want, uint32_t in_cnt) {
    const float zk = key_logit(key);
    // all that take part: up to the border there was, if it lies at this logit
    int cid = zk == w.zc ? w.cid : INT32_MAX;
    if (want < in_cnt) {
        const Weigher was = w;
        const Found f = descend<false>(
            sm,
            [&](auto fn) {
                candidates(row, sm, listed, [&](float z, int id) {
                    if (z == zk && was.above(z, id)) fn((uint32_t)id, [] { return 0.0; });
                });
            },
            16, 0, want, 0.0, false);
        cid = (int)f.ord;
    }
    w.zc = zk;
    w.cid = cid;
}

// The border of top-p among the candidates: where their running weight reaches
// goal.  False if it does not.
template <sv_dtype DT, int NT, class In>
__device__ __forceinline__ bool cut_mass(const Row<DT, NT>& row, Smem<NT>& sm, bool listed, Weigher& w,
                                         double goal, In in) {
    const Found f = descend<true>(
        sm,
        [&](auto fn) {
            candidates(row, sm, listed, [&](float z, int id) {
                if (in(z) && w.above(z, id)) fn(~order_key(z), [&] { return w.raw(z); });
            });
        },
        24, kLowDigit<DT>, 0, goal, false);
    if (!f.found) return false;
    const uint32_t key = ordinal_key<DT>(f.ord);
    const double one = w.raw(key_logit(key));
    double want = one > 0.0 ? ceil((goal - f.before.value()) / one) : 1.0;
    want = fmin(fmax(want, 1.0), (double)f.in_cnt);
    cut_ties(row, sm, listed, w, key, (uint32_t)want, f.in_cnt);
    return true;
}

// The law by digits: any settings, any row.  lb: no id below it matters;
// listed: the ids from lb up are in sm.list; m, it: the weigher's.  Not inlined:
// few rows need it, and the others' code stays small.  It and its like take and
// return their structures by value, in registers: by reference they would live
// in memory on every row's path.
template <sv_dtype DT, int NT>
__device__ __attribute__((noinline)) Result find_by_digits(const Row<DT, NT> row, const Settings set,
                                                           Smem<NT>& sm, float lb, bool listed,
                                                           double m, double it) {
    Result r{};
    Weigher w{m, it, 0.0, -kInf, -1};
    const bool use_p = set.p < 1.0f;
    const auto in = [&](float z) { return z >= lb && z > -kInf; };
    if (set.k > 0) {
        const Found f = descend<false>(
            sm,
            [&](auto fn) {
                candidates(row, sm, listed, [&](float z, int id) {
                    if (in(z)) fn(~order_key(z), [] { return 0.0; });
                });
            },
            24, kLowDigit<DT>, (uint32_t)set.k, 0.0, false);
        if (f.found)
            cut_ties(row, sm, listed, w, ordinal_key<DT>(f.ord), (uint32_t)set.k - f.before_cnt,
                     f.in_cnt);
    }
    if (use_p) {
        double total;
        int n;
        if (listed) {
            total = sum_list(sm, w, n, [&](float z, int id, double) { return w.above(z, id); });
        } else {
            double part = 0.0;
            row.each([&](float z, int id) { part += w.above(z, id) ? w.raw(z) : 0.0; });
            total = block_sum(part, sm);
        }
        cut_mass(row, sm, listed, w, (double)set.p * total, in);
    }
    w.s = (double)set.s;
    r.w = w;
    if (listed) {
        r.total = sum_list(sm, w, r.n, [&](float z, int id, double x) {
            return w.above(z, id) && x >= w.s;
        });
    }
    r.where = listed ? kListed : kInRow;
    return r;
}

// cut_mass over the list, not inlined (rarely needed).
struct Cut {
    Weigher w;
    int found;
};
template <sv_dtype DT, int NT>
__device__ __attribute__((noinline)) Cut cut_listed(const Row<DT, NT> row, Smem<NT>& sm,
                                                    const Weigher w, double goal) {
    Cut c{w, 0};
    c.found = cut_mass(row, sm, true, c.w, goal, [](float) { return true; });
    return c;
}

// Top-p's border among the ids near it, once it is known where to look: side(z)
// is 0 for logits ahead of it, 1 for those next to it, 2 behind; none of side 0
// or 1 lies below edge.  Sums the ids ahead by wave, in id order, and gathers,
// ranks and adds those near.  False, with nothing decided, where these do not
// fit the list or the border is not among them.
template <sv_dtype DT, int NT, class Side>
__device__ __forceinline__ bool finish_nucleus(const Row<DT, NT>& row, const Settings& set,
                                               Smem<NT>& sm, Result& r, double goal, float edge,
                                               Side side) {
    Weigher w = r.w;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __syncthreads();
    if (threadIdx.x == 0) sm.list_n = 0;
    __syncthreads();
    int n = 0;
    double part = 0.0;
    compact(row, sm, wave, [&](float z) { return z >= edge; }, [&](float z, int id) {
        const int s = side(z);
        n += __popcll(__ballot(s == 0));
        if (s == 0) {
            part += w.raw(z);
        } else if (s == 1 && z > -kInf) {
            const int i = atomicAdd(&sm.list_n, 1);
            if (i < kList) sm.list[i] = entry(order_key(z), id);
        }
    });
    // every lane of a wave holds the wave's count
    n = block_sum(lane == 0 ? n : 0, sm);
    const double above = block_sum(part, sm);
    const int listed = sm.list_n;
    if (listed > kList || listed == 0 || above >= goal) return false;
    // the waves' sums, kept over the search
    double mine = 0.0;
    if (threadIdx.x < NT / kWave) mine = sm.redd[threadIdx.x];
    __syncthreads();
    if (listed <= kRank) {
        rank_list(w, sm, listed);
        const int last = first_of(sm, listed, [&](int i) { return above + sm.prefix[i] >= goal; });
        if (last == listed) return false;
        w.zc = key_logit(entry_key(sm.sorted[last]));
        w.cid = entry_id(sm.sorted[last]);
    } else {
        const Cut cut = cut_listed(row, sm, w, goal - above);
        if (!cut.found) return false;
        w = cut.w;
    }
    w.s = (double)set.s;
    r.w = w;
    r.where = kInRow;
    r.n = 0;
    if (w.raw(w.zc) < w.s) return true;  // min-p cuts further: summed by the caller
    // the listed ids that stay, added to their waves' sums
    __syncthreads();
    if (threadIdx.x < NT / kWave) sm.hi[threadIdx.x] = sm.lo[threadIdx.x] = 0;
    if (threadIdx.x == 0) sm.second = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < listed; i += NT) {
        const float z = key_logit(entry_key(sm.list[i]));
        const int id = entry_id(sm.list[i]);
        if (!w.above(z, id)) continue;
        const int v = row.wave_of(id);
        const Mass q = to_mass(w.raw(z));
        atomicAdd(&sm.hi[v], q.hi);
        atomicAdd(&sm.lo[v], q.lo);
        atomicAdd(&sm.second, 1);
    }
    __syncthreads();
    if (threadIdx.x < NT / kWave)
        sm.redd[threadIdx.x] = mine + Mass{sm.hi[threadIdx.x], sm.lo[threadIdx.x]}.value();
    __syncthreads();
    r.n = n + sm.second;
    r.total = 0.0;
    for (int v = 0; v < NT / kWave; ++v) r.total += sm.redd[v];
    return true;
}

// by_value() counts the 16 octaves of magnitude up to `most`, of either sign,
// from this bf16 magnitude on.  At least 1: 0 and -0 are one logit, and in the
// list of smaller ones they are.
__device__ __forceinline__ uint32_t value_base(float most) {
    return (uint32_t)max((int)(__float_as_uint(most) >> 16) + 1 - (kValues - 1), 1);
}
// The largest magnitude that matters: 2^(-65) of the largest weight lies 45 T
// below it.
__device__ __forceinline__ float value_reach(float m, float t) {
    return fmaxf(fabsf(m), fabsf(m - 45.0f * t));
}

template <int NT>
__device__ __forceinline__ void clear_values(Smem<NT>& sm) {
    for (int i = threadIdx.x; i < 2 * kValues; i += NT) sm.value[i] = 0;
    if (threadIdx.x == 0) sm.list_n = 0;
    __syncthreads();
}

// Counts a granule's values, positive ones by magnitude and behind them negative
// ones (values out of range behind both, a place for each lane), and lists the
// ids of magnitudes below the range.
template <int NT>
__device__ __forceinline__ void count_values(const typename Row<SV_BF16, NT>::Raw& g, int id0,
                                             Smem<NT>& sm, uint32_t base) {
    const uint32_t out = 2 * kValues + (threadIdx.x & 63);
    u16x2 least{0xffff, 0xffff};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t mags = g.w[i] & 0x7fff7fffu;
        least = __builtin_elementwise_min(least, __builtin_bit_cast(u16x2, mags));
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const uint32_t at = (half ? mags >> 16 : mags & 0xffffu) - base;
            const uint32_t negative = (g.w[i] >> (half ? 31 : 15)) & 1u;
            atomicAdd(&sm.value[at < (uint32_t)kValues ? at + negative * kValues : out], 1u);
        }
    }
    if (min(least.x, least.y) >= base) return;
    float z[8];
    g.unpack(z);
    const float below = __uint_as_float(base << 16);
    int c = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) c += fabsf(z[e]) < below ? 1 : 0;
    int at = atomicAdd(&sm.list_n, c);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (fabsf(z[e]) < below) {
            if (at < kRank) sm.list[at] = entry(order_key(z[e]), id0 + e);
            ++at;
        }
    }
}

// The want-th lowest of the listed ids; not inlined (rarely needed).
template <int NT>
__device__ __attribute__((noinline)) int nth_id(Smem<NT>& sm, uint32_t want) {
    return (int)descend<false>(
               sm,
               [&](auto fn) {
                   for (int i = threadIdx.x; i < sm.list_n; i += NT)
                       fn((uint32_t)entry_id(sm.list[i]), [] { return 0.0; });
               },
               16, 0, want, 0.0, false).ord;
}

// The sum of a bf16 row's weights, and top-p's border, from how many ids have
// each value: one LDS add an id (8 clocks a wave) where a weight takes 21 fp64
// operations, then one weight a value (129,280 ids: 24 us for the pass that sums
// them by id, 7 us this way).  The values counted are the 16 octaves up to the
// largest magnitude that matters, of either sign; the few ids of smaller ones
// are listed and ranked; larger negative ones weigh less than 2^-64 and add
// nothing.  base: where the values that pass 1 counted begin, 0 if it counted
// none; they are counted again if they do not reach far enough.  Sets r.total,
// and for top-p the border and r.n; where a draw follows, the waves' sums too
// (finish_nucleus).  False, with nothing decided, where the list does not hold
// the small ones or the border's ties.
template <bool DRAWS, int NT>
__device__ __forceinline__ bool by_value(const Row<SV_BF16, NT>& row, const Settings& set,
                                         Smem<NT>& sm, Result& r, uint32_t base) {
    Weigher w = r.w;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float most = value_reach((float)w.m, set.t);
    if (!(most < 1e38f)) return false;
    const uint32_t exact = value_base(most);
    if (base < exact || (base > exact && sm.list_n > kRank)) {
        base = exact;
        __syncthreads();
        clear_values(sm);
        row.each_granule([&](const typename Row<SV_BF16, NT>::Raw& g, int id0) {
            count_values(g, id0, sm, base);
        });
        __syncthreads();
    }
    const int small = sm.list_n;
    if (small > kRank) return false;
    rank_list(w, sm, small);
    const double small_mass = small > 0 ? sm.prefix[small - 1] : 0.0;
    // each thread's share of the values, in descending order (positive ones from
    // the largest down, then negative ones from the smallest magnitude up), and
    // what is ahead of it
    constexpr int kEach = 2 * kValues / NT;
    double mass[kEach], own = 0.0;
    uint32_t cnt[kEach], own_cnt = 0;
    const auto logit = [&](int o) {
        const uint32_t mag = base + (uint32_t)(o < kValues ? kValues - 1 - o : o - kValues);
        return __uint_as_float((mag << 16) | (o < kValues ? 0u : 0x80000000u));
    };
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int o = kEach * (int)threadIdx.x + i;
        cnt[i] = sm.value[o < kValues ? kValues - 1 - o : o];
        mass[i] = cnt[i] ? (double)cnt[i] * w.raw(logit(o)) : 0.0;
        own += mass[i];
        own_cnt += cnt[i];
    }
    const double incl = wave_incl_sum_dpp(own, lane);
    const uint32_t incl_cnt = wave_incl_sum_dpp(own_cnt, lane);
    if (lane == 63) {
        sm.redd[wave] = incl;
        sm.red[wave] = incl_cnt;
    }
    if (threadIdx.x == 0) sm.first = -1;
    __syncthreads();
    double before = incl - own, total = small_mass;
    uint32_t before_cnt = incl_cnt - own_cnt;
    for (int v = 0; v < NT / kWave; ++v) {
        if (v < wave) before += sm.redd[v], before_cnt += sm.red[v];
        total += sm.redd[v];
    }
    r.total = total;
    if (set.p >= 1.0f) return true;
    // the border: a value, or one of the small ids
    const double goal = (double)set.p * total;
    const bool negative = kEach * (int)threadIdx.x >= kValues;
    if (negative) before += small_mass, before_cnt += small;
    double at_mass = 0.0;
    uint32_t at_cnt = 0;
    int found = -1;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (found < 0 && cnt[i] != 0 && before + mass[i] >= goal) {
            found = i;
            at_mass = before;
            at_cnt = before_cnt;
        }
        before += mass[i];
        before_cnt += cnt[i];
    }
    // positive bins end where the small ids begin
    if (threadIdx.x == kValues / kEach - 1) sm.before.hi = __double_as_longlong(before), sm.cnt[0] = before_cnt;
    const int thread = first_of(sm, NT, [&](int) { return found >= 0; });
    const double positive = __longlong_as_double((long long)sm.before.hi);
    const int in_small = first_of(sm, small, [&](int i) { return positive + sm.prefix[i] >= goal; });
    if (in_small < small && thread >= kValues / kEach) {
        w.zc = key_logit(entry_key(sm.sorted[in_small]));
        w.cid = entry_id(sm.sorted[in_small]);
        r.n = (int)sm.cnt[0] + in_small + 1;
        r.total = positive + sm.prefix[in_small];
    } else {
        if (thread >= NT) return false;
        if ((int)threadIdx.x == thread) {
            uint32_t n = 0;
            double x = 0.0;
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (i == found) n = cnt[i], x = mass[i];
            const float z = logit(kEach * thread + found);
            const double one = w.raw(z);
            double want = one > 0.0 ? ceil((goal - at_mass) / one) : 1.0;
            want = fmin(fmax(want, 1.0), (double)n);
            sm.digit = order_key(z);
            sm.before_cnt = (uint32_t)want;
            sm.in_cnt = n;
            sm.first = (int)at_cnt;
            sm.before.lo = __double_as_longlong(want == (double)n ? at_mass + x : at_mass + want * one);
        }
        __syncthreads();
        const uint32_t want = sm.before_cnt, n = sm.in_cnt;
        w.zc = key_logit(sm.digit);
        if constexpr (DRAWS) {
            const float zc = w.zc;
            return finish_nucleus(row, set, sm, r, goal, zc,
                                  [zc](float z) { return z > zc ? 0 : 1; });
        }
        r.n = sm.first + (int)want;
        r.total = __longlong_as_double((long long)sm.before.lo);
        __syncthreads();
        if (want == n) {
            w.cid = INT32_MAX;
        } else {
            // the want-th lowest id of the border's value
            if (n > (uint32_t)kList) return false;
            if (threadIdx.x == 0) sm.list_n = 0;
            __syncthreads();
            const uint32_t at = __float_as_uint(w.zc), both = at | at >> 16;
            row.template granules<8>(
                [&](const typename Row<SV_BF16, NT>::Raw& g, int id0) {
                    // whether some half word equals zc's (or may)
                    uint32_t some = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t x = g.w[i] ^ both;
                        some |= (x - 0x00010001u) & ~x;
                    }
                    if ((some & 0x80008000u) == 0) return;
                    float z[8];
                    g.unpack(z);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (z[e] == w.zc) {
                            const int i = atomicAdd(&sm.list_n, 1);
                            if (i < kList) sm.list[i] = entry(sm.digit, id0 + e);
                        }
                },
                [](int) {});
            __syncthreads();
            if (n <= (uint32_t)kRank) {
                rank_list(w, sm, (int)n);
                w.cid = entry_id(sm.sorted[want - 1]);
            } else {
                w.cid = nth_id(sm, want);
            }
        }
    }
    w.s = (double)set.s;
    // min-p cuts further, or the waves' sums are wanted: summed by the caller
    if (DRAWS || w.raw(w.zc) < w.s) r.n = 0;
    r.w = w;
    r.where = kInRow;
    return true;
}

// Steps of the weight, from a logit that is about the row's largest: kPerOctave
// for each factor of 2, the first kAbove of them above it.
struct Steps {
    float ref, per_logit;
    // the step's number, with the place within it; monotone in z, whatever it
    // rounds to
    __device__ __forceinline__ float at(float z) const {
        const float v = (ref - z) * per_logit + (float)kAbove;
        return fminf(fmaxf(v, 0.0f), (float)(kSteps - 1));
    }
    __device__ __forceinline__ int of(float z) const { return (int)at(z); }
};

template <int NT>
__device__ __forceinline__ void clear_steps(Smem<NT>& sm) {
    for (int i = threadIdx.x; i < kSteps; i += NT) sm.step[i] = 0;
    __syncthreads();
}

// The histogram only says where to look.  An id adds its weight over the step's
// largest (between 1 and 2^(-1/32), linear within 3e-5) in units of 1/1024: at
// most 2^30 a step; the last step's, of next to no weight, are left out.  (LDS
// adds in fp32 took 170 clocks a wave here, 64-bit integer ones 31.)
template <int NT>
__device__ __forceinline__ void count_step(Smem<NT>& sm, const Steps& steps, float z) {
    const float v = steps.at(z), f = v - floorf(v);
    if (v < (float)(kSteps - 1))
        atomicAdd(&sm.step[(int)v], (uint32_t)fmaf(f, -1024.0f * (1.0f - 0.978572f), 1024.5f));
}

// Top-p alone.  steps: of the histogram that pass 1 made, total: the sum it took
// of the row's weights (not made: both are made here).  Returns false, with
// nothing decided, where the ids next to the border do not fit the list.
template <sv_dtype DT, int NT>
__device__ __forceinline__ bool find_nucleus(const Row<DT, NT>& row, const Settings& set, Smem<NT>& sm,
                                             Result& r, Steps steps, double total, bool made) {
    Weigher w = r.w;
    if (!made) {
        steps.ref = (float)w.m;
        clear_steps(sm);
        double part = 0.0;
        row.each([&](float z, int id) {
            part += w.raw(z);  // -inf: 0
            count_step(sm, steps, z);
        });
        total = block_sum(part, sm);
    }
    const double above = w.raw(steps.ref);  // of the largest weight
    const double goal = (double)set.p * total;
    // The border is where the weight behind it falls to total - goal; taken
    // from that side, a histogram off by 2^-11 of what it holds is off by
    // little where top-p leaves little out.
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    constexpr int kEach = kSteps / NT;  // steps a thread adds up
    double mass[kEach], own = 0.0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int s = kEach * threadIdx.x + i;
        mass[i] = (double)sm.step[s] * above *
                  (pow2((double)(kAbove - s) / (double)kPerOctave) * 0x1p-10);
        own += mass[i];
    }
    const double incl = wave_incl_sum_dpp(own, lane);
    __syncthreads();
    if (lane == 63) sm.redd[wave] = incl;
    if (threadIdx.x == 0) sm.first = sm.second = kSteps - 1, sm.list_n = 0;
    __syncthreads();
    double before = incl - own, all = 0.0;
    for (int v = 0; v < NT / kWave; ++v) {
        if (v < wave) before += sm.redd[v];
        all += sm.redd[v];
    }
    const double left = total - goal, off = 6e-4 * left + 1e-12 * total;
    double behind = all - before;  // the weight from a step on
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int s = kEach * threadIdx.x + i;
        const double next = behind - mass[i];
        if (next - off <= left && (s == 0 || behind - off > left)) sm.first = s;
        if (next + off <= left && (s == 0 || behind + off > left)) sm.second = s;
        behind = next;
    }
    __syncthreads();
    const int b1 = sm.first, b2 = sm.second;
    // logits of step b2 or less: at least this one, or a little below
    const float down = (float)(b2 + 1 - kAbove) / steps.per_logit;
    const float edge = steps.ref - down - (fabsf(down) * 1e-5f + 1e-3f / steps.per_logit) -
                       fabsf(steps.ref) * 1e-6f;
    return finish_nucleus(row, set, sm, r, goal, edge, [&](float z) {
        const int s = steps.of(z);
        return s < b1 ? 0 : s <= b2 ? 1 : 2;
    });
}

// DRAWS: a draw follows, which needs the waves' sums (sm.redd) where the law is
// found again in the row; without it r.n of a row that nothing cuts is not set.
template <bool DRAWS, sv_dtype DT, int NT>
__device__ __forceinline__ Result find_law(const Row<DT, NT>& row, const Settings& set, Smem<NT>& sm) {
    using Raw = typename Row<DT, NT>::Raw;
    // granules of a batch of loads: 128 bytes a lane in flight
    constexpr int kAhead = 16 / Row<DT, NT>::kBytes;
    const int lane = threadIdx.x & 63;
    Result r{};
    // Pass 1: largest logit, faults; and where nothing but top-p may cut, what
    // needs every id, taken relative to the largest of the first ids: the values
    // of a bf16 row that by_value() decides, in a range twice as far as that one
    // asks for; else the sum of the weights, by wave, and top-p's histogram.
    // Loads in flight while values are counted: eight without a draw (verification
    // of 256 x 7 rows under top-p: 308 us, 313 with four, 331 with two); two with
    // one, where more make the kernel's other ways slower (2048 rows, greedy: 94
    // us, 104 with four or eight; top-k: 127, 144 and 143) than top-p gains (341,
    // 327 and 327).  Two of bf16 and four of fp32 while weights are summed: twice
    // or four times as many measured the same within 3 %.
    const bool use_p = set.p < 1.0f;
    Extremes<DT> ex, batch;
    uint32_t base = 0;
    bool made = false;
    float ref = 0.0f;
    double part = 0.0;
    int n_part = 0;
    Weigher& w = r.w;
    w.it = set.t == 0.0f ? 0.0 : kLog2e64 / (double)set.t;
    Steps steps{0.0f, fminf(kPerOctave * (float)w.it, 1e30f)};
    if (!set.bad && set.k == 0 && set.t > 0.0f && (use_p || set.s == 0.0f)) {
        Extremes<DT> first;
        const Raw g = row.raw(row.turn_id(0));
#pragma unroll
        for (int i = 0; i < Row<DT, NT>::kWords; ++i) first.add(g.w[i]);
        ref = key_logit(block_max(first.top(), sm));
        if constexpr (DT == SV_BF16) {
            const float most = 2.0f * value_reach(ref, set.t);
            if ((use_p || !DRAWS) && most < 1e38f) {
                base = value_base(most);
                clear_values(sm);
                row.template granules<DRAWS ? 2 : 8>(
                    [&](const Raw& g, int id0) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) ex.add(g.w[i]);
                        count_values(g, id0, sm, base);
                    },
                    [](int) {});
            }
        }
        if (base == 0 && is_finite_bits(ref)) {
            made = true;
            steps.ref = ref;
            w.m = (double)ref;
            const Weigher law = w;
            if (use_p) clear_steps(sm);
            row.template in_order<kAhead / (DT == SV_BF16 ? 4 : 1)>([&](const Raw& g, int) {
                float z[8];
                g.unpack(z);
#pragma unroll
                for (int i = 0; i < Row<DT, NT>::kWords; ++i) ex.add(g.w[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    part += law.raw(z[e]);
                    if (use_p) count_step(sm, steps, z[e]);
                    else n_part += __popcll(__ballot(z[e] > -kInf));
                }
            });
        }
    }
    if (base == 0 && !made) {
        row.template granules<kAhead>(
            [&](const Raw& g, int) {
#pragma unroll
                for (int i = 0; i < 2 * Row<DT, NT>::kBytes; ++i) batch.add(g.w[i]);
            },
            [&](int b) {
                if (b < Smem<NT>::kBatches)
                    sm.batch_top[b][threadIdx.x] = (uint16_t)(batch.top() >> 16);
                ex.add(batch);
                batch = Extremes<DT>{};
            });
    }
    const uint32_t mine = ex.top();
    const uint32_t top = block_max(mine, sm);
    const int bad = __syncthreads_or(ex.bad());
    if (bad || top <= kMinusInfKey) r.fault |= SV_DEV_NONFINITE;
    if (set.bad) r.fault |= SV_DEV_BAD_PARAM;
    if (r.fault) return r;
    w.m = (double)key_logit(top);
    w.s = 0.0;
    w.zc = -kInf;
    w.cid = -1;  // no id of -inf counts

    // lb: no id below this logit is in the support (nor, with top-k, among
    // the first k)
    float lb = -kInf;
    if (set.t == 0.0f) {
        lb = key_logit(top);
    } else if (set.k > 0 && set.k <= NT) {
        // Just below the k-th largest of the threads' maxima: k ids are at
        // least that.  Bins of 2^16 key steps (a bf16 step) below the largest
        // logit; where fewer than k maxima are in the first 255, no bound.
        const uint32_t bin = min((top - mine) >> 16, 255u);
        const Found f = descend<false>(
            sm, [&](auto fn) { if (mine > kMinusInfKey) fn(bin, [] { return 0.0; }); }, 0, 0,
            (uint32_t)set.k, 0.0, false);
        const uint32_t below = (f.ord + 1) << 16;
        if (f.found && f.ord < 255 && top - kMinusInfKey > below) lb = key_logit(top - below + 1);
    }
    if (set.s > 0.0f && set.t > 0.0f && !(use_p && set.k > 0)) {
        // a little below m + T ln s, for the roundings on the way (of the
        // logits' size, and of an exponent's: weights next to 1 round to 1)
        const double z = w.m + log((double)set.s) * (double)set.t;
        const double slack = 1e-6 * (fabs(w.m) + fabs(z) + (double)set.t);
        lb = fmaxf(lb, (float)(z - slack));
    }
    // Sums relative to a logit so far below the largest that the histogram, or
    // the exponents, do not reach it are taken again.  (Of 256 rows some lie 8
    // octaves off, and the slowest counts.)
    if (made && (w.m - (double)ref) * w.it > (use_p ? (double)kAbove / (double)kPerOctave : 500.0))
        made = false;
    double total = 0.0;
    if (made) {
        part *= w.raw(ref);
        total = block_sum(part, sm);
        if (!use_p) {  // nothing is cut
            r.n = block_sum(lane == 0 ? n_part : 0, sm);
            r.total = total;
            r.where = kInRow;
            return r;
        }
    }
    bool decided = false;
    if (set.k == 0 && set.t > 0.0f) {
        if constexpr (DT == SV_BF16) {
            // the border, and without a draw everything, by the row's values
            if (use_p || (!DRAWS && set.s == 0.0f)) decided = by_value<DRAWS>(row, set, sm, r, base);
            if (decided && (r.n > 0 || !use_p)) return r;
        }
        if (!decided && use_p) {
            decided = find_nucleus(row, set, sm, r, steps, total, made);
            if (decided && r.n > 0) return r;
        }
        if (use_p) lb = -kInf;
    }
    // keep what is left in LDS if it fits
    bool listed = lb > -kInf;
    if (listed) {
        if (threadIdx.x == 0) sm.list_n = 0;
        __syncthreads();
        // A thread whose own maximum is below the bound has none; the others
        // look at their batches whose maximum is not, which of the granules
        // hold one, and read those again.  (Code that is run once is paid for
        // in instruction fetches: none of it unrolled.)
        if (mine >= order_key(lb)) {
            const uint32_t least = order_key(lb) >> 16;
            for (int s0 = 0; s0 < row.turns(); s0 += kAhead) {
                const int b = s0 / kAhead;
                if (b < Smem<NT>::kBatches && sm.batch_top[b][threadIdx.x] < least) continue;
                unsigned hits = 0;
                Raw g[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    g[i] = row.fetch(min(row.turn_id(s0 + i), row.vocab));
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    float z[8];
                    g[i].unpack(z);
                    float big = z[0];
#pragma unroll
                    for (int e = 1; e < 8; ++e) big = fmaxf(big, z[e]);
                    // a granule past the row's end shows its last ids: looked
                    // at again below
                    if (big >= lb && row.turn_id(s0 + i) < row.vocab) hits |= 1u << i;
                }
#pragma unroll 1
                for (; hits != 0; hits &= hits - 1) {
                    const int id0 = row.turn_id(s0 + __builtin_ctz(hits));
                    float z[8];
                    row.raw(id0).unpack(z);
                    int c = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) c += z[e] >= lb ? 1 : 0;
                    int at = atomicAdd(&sm.list_n, c);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (z[e] >= lb) {
                            if (at < kList) sm.list[at] = entry(order_key(z[e]), id0 + e);
                            ++at;
                        }
                    }
                }
            }
        }
        __syncthreads();
        listed = sm.list_n <= kList;
    }
    if (listed && sm.list_n <= kRank) {
        const int all = sm.list_n;
        rank_list(w, sm, all);
        int n = set.k > 0 ? min(set.k, all) : all;
        if (use_p) {
            const double goal = (double)set.p * sm.prefix[n - 1];
            n = min(n, first_of(sm, n, [&](int i) { return sm.prefix[i] >= goal; }) + 1);
        }
        if (set.s > 0.0f)
            n = max(1, first_of(sm, n, [&](int i) { return sm.weight[i] < (double)set.s; }));
        if (set.t == 0.0f) n = 1;
        w.zc = key_logit(entry_key(sm.sorted[n - 1]));
        w.cid = entry_id(sm.sorted[n - 1]);
        r.n = n;
        r.total = sm.prefix[n - 1];
        r.where = kRanked;
        return r;
    }
    if (set.t == 0.0f) {
        // more than kRank ids of the largest logit: the lowest
        uint32_t first = 0;
        row.each([&](float z, int id) { if (z >= lb) first = max(first, ~(uint32_t)id); });
        first = block_max(first, sm);
        w.zc = lb;
        w.cid = (int)~first;
        if (threadIdx.x == 0) sm.sorted[0] = entry(top, w.cid);
        __syncthreads();
        r.n = 1;
        r.total = 1.0;
        r.where = kRanked;
        return r;
    }
    r.where = kInRow;
    if (!decided) {
        if (use_p || set.k > 0 || listed)
            r = find_by_digits<DT, NT>(row, set, sm, lb, listed, w.m, w.it);
        if (r.where == kListed) return r;
    }
    r.w.s = (double)set.s;
    // how many, and their weight; leaves the waves' sums in sm.redd
    const Weigher law = r.w;
    int n = 0;
    double mass = 0.0;
    if (law.zc == -kInf && law.s == 0.0) {
        row.each([&](float z, int id) {
            n += __popcll(__ballot(z > -kInf));
            mass += law.raw(z);
        });
    } else {
        compact(row, sm, threadIdx.x >> 6, [&](float z) { return z >= law.zc && z >= lb; }, [&](float z, int id) {
            const double x = law.raw(z);
            const bool live = law.above(z, id) && x >= law.s;
            n += __popcll(__ballot(live));
            mass += live ? x : 0.0;
        });
    }
    r.n = block_sum(lane == 0 ? n : 0, sm);
    r.total = block_sum(mass, sm);
    return r;
}

// The smallest id whose running sum, over a row in segments, passes goal.  sums
// holds the sum of each of the `segments`; all waves together sum the steps of
// the segment that holds the crossing, one wave walks the step that does.
// first_id(segment, step, lane) is a lane's first id, weights(id0, x) gives the
// 8 weights at ids id0 .. id0 + 7.  If rounding leaves no such id, the last one
// of positive weight.
template <int NT, class Weights, class FirstId>
__device__ __forceinline__ int walk_row(Smem<NT>& sm, const double* sums, int segments, double goal, int steps,
                        FirstId first_id, int vocab, Weights weights) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    double before = 0.0;
    int owner = -1;
    for (int w = 0; w < segments; ++w) {
        if (before + sums[w] > goal) {
            owner = w;
            break;
        }
        before += sums[w];
    }
    if (owner < 0) {
        goal = kInf;
        before = 0.0;
        for (int w = 0; w < segments; ++w)
            if (sums[w] > 0.0) owner = w;
    }
    const auto read = [&](int s, double* x) {
        const int id0 = first_id(owner, s, lane);
        double mine = 0.0;
        if (id0 < vocab) {
            weights(id0, x);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = 0.0;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) mine += x[e];
        return mine;
    };
    // all waves sum the segment's steps; a wave keeps its last one's weights
    double x[8], incl = 0.0;
    int held = -1;
    for (int s = wave; s < steps; s += NT / kWave) {
        incl = wave_incl_sum_dpp(read(s, x), lane);
        held = s;
        if (lane == 63) sm.seg[s] = incl;
    }
    __syncthreads();
    int step = -1, positive = 0;
    double at = before;
    for (int s = 0; s < steps; ++s) {
        const double sum = sm.seg[s];
        if (sum > 0.0) positive = s;
        if (step < 0 && before + sum > goal) {
            step = s;
            at = before;
        }
        before += sum;
    }
    if (step < 0) {
        step = positive;
        goal = kInf;
    }
    if (wave == step % (NT / kWave)) {
        if (held != step) incl = wave_incl_sum_dpp(read(step, x), lane);
        const int id0 = first_id(owner, step, lane);
        double mine = 0.0;
#pragma unroll
        for (int e = 0; e < 8; ++e) mine += x[e];
        double c = at + (incl - mine);
        int hit = -1, last = -1;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            c += x[e];
            if (x[e] > 0.0) last = id0 + e;
            if (hit < 0 && x[e] > 0.0 && c > goal) hit = id0 + e;
        }
        const unsigned long long hits = __ballot(hit >= 0), some = __ballot(last >= 0);
        int tok = 0;
        if (hits) tok = __builtin_amdgcn_readlane(hit, __builtin_ctzll(hits));
        else if (some) tok = __builtin_amdgcn_readlane(last, 63 - __builtin_clzll(some));
        if (lane == 0) sm.redi[0] = tok;
    }
    __syncthreads();
    return sm.redi[0];
}

// A draw over the listed ids, digit by digit of the id; not inlined (rarely
// needed).
template <sv_dtype DT, int NT>
__device__ __attribute__((noinline)) int draw_listed(const Row<DT, NT> row, Smem<NT>& sm,
                                                     const Weigher w, float u, double goal) {
    const auto live = [&](auto fn) {
        candidates(row, sm, true, [&](float z, int id) {
            const double x = w(z, id);
            if (x > 0.0) fn((uint32_t)id, [&] { return x; });
        });
    };
    // u = 0: the lowest id of any weight, however small
    if (u == 0.0f) return (int)descend<false>(sm, live, 16, 0, 1, 0.0, false).ord;
    return (int)descend<true>(sm, live, 16, 0, 0, goal, true).ord;
}

// The id a uniform u in [0, 1) draws from a law find_law has just made.
template <sv_dtype DT, int NT>
__device__ __forceinline__ int draw(const Row<DT, NT>& row, const Result& r, float u, Smem<NT>& sm) {
    const double goal = (double)u * r.total;
    if (r.where == kRanked) {
        if (r.n == 1) return entry_id(sm.sorted[0]);
        // running sums over ascending ids: each thread adds, in rank order,
        // the weights of the ids up to its own
        const int i = threadIdx.x;
        uint32_t past = 0, mine = 0;  // ~id of a thread's own id if it is drawn past
        if (i < r.n && sm.weight[i] > 0.0) {
            mine = (uint32_t)sm.sorted[i];
            double c = 0.0;
#pragma unroll 8
            for (int j = 0; j < r.n; ++j)
                c += (uint32_t)sm.sorted[j] >= mine ? sm.weight[j] : 0.0;
            if (c > goal) past = mine;
        }
        past = block_max(past, sm);
        if (past != 0) return (int)~past;
        return (int)block_max(mine != 0 ? ~mine : 0u, sm);  // rounding left none: the last id
    }
    if (r.where == kInRow) {
        return walk_row(
            sm, sm.redd, NT / kWave, goal, row.steps,
            [&](int w, int s, int l) { return row.first_id(w, s, l); }, row.vocab,
            [&](int id0, double* x) {
                float z[8];
                row.load(id0, z);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = r.w(z[e], id0 + e);
            });
    }
    return draw_listed(row, sm, r.w, u, goal);
}

}  // namespace law
}  // namespace sv
