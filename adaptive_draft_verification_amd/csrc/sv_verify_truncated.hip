// sv_verify_truncated: verification of the kept rows under truncated laws
// (temperature, top-k, top-p, min-p of each request; sv_law.h).  The rule is
// sv_verify's (rejection sampling keeps the target's law), with p and q the
// truncated laws.
//
// Launch 1, one 512-thread workgroup per row slot: the law of each target row
// 0 .. b and draft row 0 .. b - 1 of a request (LawRecord), and the weight it
// gives the position's draft id.  From these a wave decides (lane j: position
// j).  Launch 2: the row or two rows that decide the token at L are summed in
// eight parts, in 64 bits.  Launch 3: the outputs, and the draw: the part that
// holds the crossing is summed again by segments and steps, one step is walked.
#include "sv_law.h"
#include "sv_launch.h"

namespace sv {
namespace {

template <sv_dtype DT>
constexpr int kBytes = DT == SV_BF16 ? 2 : 4;

struct Span {
    int lo, b;
    bool ok;
};

__device__ __forceinline__ Span span(const VerifyTruncatedArgs& a, int r) {
    const int lo = a.cu_rows[r], hi = a.cu_rows[r + 1];
    const int64_t b = (int64_t)hi - lo - 1;
    return {lo, (int)b, lo >= 0 && b >= 0 && b <= a.k_max && hi <= a.target_rows};
}

template <sv_dtype DT>
__device__ __forceinline__ const char* target_row(const VerifyTruncatedArgs& a, int lo, int j) {
    return static_cast<const char*>(a.target) +
           ((int64_t)lo + j) * a.target_ld * kBytes<DT>;
}
template <sv_dtype DT>
__device__ __forceinline__ const char* draft_row(const VerifyTruncatedArgs& a, int r, int j) {
    return static_cast<const char*>(a.draft) +
           ((int64_t)r * a.k_max + j) * a.draft_ld * kBytes<DT>;
}

// grid: position-major, so that the slots past a request's rows, which exit at
// once, come last
template <sv_dtype DT, int kLaws>
__global__ __launch_bounds__(kLaws, kLaws == kWave ? 1 : 4) void laws_kernel(VerifyTruncatedArgs a) {
    __shared__ law::Smem<kLaws> sm;
    const int r = blockIdx.x % a.n_req, slot = blockIdx.x / a.n_req;
    const bool is_draft = slot & 1;       // target 0, draft 0, target 1, ...
    const int j = slot >> 1;
    const Span s = span(a, r);
    if (!s.ok || j > s.b || (is_draft && j == s.b)) return;
    const law::Row<DT, kLaws> row(is_draft ? draft_row<DT>(a, r, j) : target_row<DT>(a, s.lo, j), a.vocab);
    const law::Settings set =
        law::settings(is_draft ? a.draft_law : a.target_law, r, a.vocab);
    const law::Result res = law::find_law<false>(row, set, sm);
    if (threadIdx.x != 0) return;
    LawRecord rec{};
    rec.fault = res.fault;
    if (!res.fault) {
        rec.total = res.total;
        rec.top = (float)res.w.m;
        rec.zc = res.w.zc;
        rec.cid = res.w.cid;
        const int d = j < s.b ? a.draft_tokens[(int64_t)r * a.k_max + j] : -1;
        if (d >= 0 && d < a.vocab) rec.drafted = res.w(row.one(d), d);
    }
    a.laws[(int64_t)r * (2 * a.k_max + 1) + (is_draft ? a.k_max + 1 + j : j)] = rec;
}

__device__ law::Weigher weigher(const LawRecord& rec, const law::Settings& set) {
    law::Weigher w;
    w.m = (double)rec.top;
    w.it = set.t == 0.0f ? 0.0 : law::kLog2e64 / (double)set.t;
    w.s = set.t == 0.0f ? 0.0 : (double)set.s;
    w.zc = rec.zc;
    w.cid = rec.cid;
    return w;
}

// A request's decisions, as one wave takes them (lane j: position j).
struct Decision {
    int L, fault;  // the same in every lane; SV_DEV_* bits
    float v;       // the draw's uniform
    bool acc;
    double p, q;   // of the lane's draft id (-1: none)
    int d;
};

__device__ __forceinline__ Decision decide(const VerifyTruncatedArgs& a, int r, const Span& s) {
    const int j = threadIdx.x & 63, k_max = a.k_max;
    const LawRecord* laws = a.laws + (int64_t)r * (2 * k_max + 1);
    Decision o{0, s.ok ? 0 : SV_DEV_BAD_CU_ROWS, 0.0f, true, -1.0, -1.0, -1};
    // settings of the draft's law matter only where a draft row is read
    if (law::settings(a.target_law, r, a.vocab).bad ||
        (s.ok && s.b > 0 && law::settings(a.draft_law, r, a.vocab).bad))
        o.fault |= SV_DEV_BAD_PARAM;
    float u = 0.0f, v = 0.0f;
    draw_uniforms(a.seed, a.step, (uint32_t)r, (uint32_t)j, &u, &v);
    if (s.ok) {
        if (j < s.b) {
            o.d = a.draft_tokens[(int64_t)r * k_max + j];
            if (o.d < 0 || o.d >= a.vocab) o.fault |= SV_DEV_BAD_TOKEN;
            const LawRecord t = laws[j], w = laws[k_max + 1 + j];
            o.fault |= t.fault | w.fault;
            if (!(t.fault | w.fault)) {
                o.p = t.drafted / t.total;
                o.q = w.drafted / w.total;
                o.acc = o.q > 0.0 ? (double)u < o.p / o.q : o.p > 0.0;
            }
        }
        if (j == 0) o.fault |= laws[s.b].fault;
    }
    o.fault = wave_or_int(o.fault);
    const uint64_t rej = __ballot(!o.acc);
    o.L = rej ? __builtin_ctzll(rej) : s.b;
    o.v = __shfl(v, o.L & 63);
    if (o.L == kWave) {
        float u2;
        draw_uniforms(a.seed, a.step, (uint32_t)r, (uint32_t)o.L, &u2, &v);
        o.v = v;
    }
    return o;
}

// The weights the token at L is drawn from: p's, or the residual's.
template <sv_dtype DT, int NT>
struct Drawn {
    law::Weigher pw, qw;
    law::Row<DT, NT> prow, qrow;
    double ip, iq;
    bool minus;  // the residual p - q, not p

    __device__ __forceinline__ Drawn(const VerifyTruncatedArgs& a, int r, const Span& s, int L,
                                     int segments)
        : prow(target_row<DT>(a, s.lo, L), a.vocab, segments),
          qrow(prow), ip(0.0), iq(0.0), minus(L < s.b) {
        const LawRecord* laws = a.laws + (int64_t)r * (2 * a.k_max + 1);
        const LawRecord pr = laws[L];
        pw = weigher(pr, law::settings(a.target_law, r, a.vocab));
        qw = pw;
        if (minus) {
            const LawRecord qr = laws[a.k_max + 1 + L];
            qw = weigher(qr, law::settings(a.draft_law, r, a.vocab));
            qrow = law::Row<DT, NT>(draft_row<DT>(a, r, L), a.vocab, segments);
            ip = 1.0 / pr.total;
            iq = 1.0 / qr.total;
        }
    }
    // z: p's logit at id
    __device__ __forceinline__ double of(float z, int id) const {
        const double x = pw(z, id);
        return minus && x > 0.0 ? fmax(0.0, x * ip - qw(qrow.one(id), id) * iq) : x;
    }
    __device__ __forceinline__ void of8(int id0, double* x) const {
        float z[8], y[8];
        prow.load(id0, z);
        if (minus) qrow.load(id0, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = pw(z[e], id0 + e);
            if (minus && x[e] > 0.0) x[e] = fmax(0.0, x[e] * ip - qw(y[e], id0 + e) * iq);
        }
    }
    // The calling wave's sum over a segment of the row, in every lane.
    __device__ __forceinline__ double sum(law::Smem<NT>& sm, int segment) const {
        double part = 0.0;
        if (pw.it == 0.0) {  // greedy: one id
            if ((pw.cid >> 3) / prow.per == segment && (threadIdx.x & 63) == 0)
                part = of(prow.one(pw.cid), pw.cid);
        } else if (pw.zc == -law::kInf) {  // nothing cut: every id weighs
            const int lane = threadIdx.x & 63;
            for (int st = 0; st < prow.steps; ++st) {
                const int id0 = prow.first_id(segment, st, lane);
                if (prow.first_id(segment, st, 0) >= prow.vocab) break;
                double x[8];
                of8(id0, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) part += x[e];
            }
        } else {
            law::compact<4>(prow, sm, segment, [&](float z) { return z >= pw.zc; },
                         [&](float z, int id) { part += of(z, id); });
        }
        return wave_sum(part);
    }
};

// The calling workgroup's segments of a part of the row, summed by its waves
// into sm.redd, and their total, the same whenever it is taken.
template <sv_dtype DT, int NT>
__device__ double sum_part(const Drawn<DT, NT>& drawn, law::Smem<NT>& sm, int part) {
    constexpr int kWaves = NT / kWave;
    const int wave = threadIdx.x >> 6;
    const double x = drawn.sum(sm, part * kWaves + wave);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sm.redd[wave] = x;
    __syncthreads();
    double total = 0.0;
    for (int w = 0; w < kWaves; ++w) total += sm.redd[w];
    return total;
}

// Launch 2: the sums of the row (or two) that decide the token at L, kParts
// workgroups a request: requests whose settings cut nothing take a hundred times
// the work of greedy ones, and would leave most CUs waiting if each had one
// workgroup (256 x 7, mixed: 129 us for this launch and the next in one, 72 in
// two).
template <sv_dtype DT, int NT, int kParts>
__global__ __launch_bounds__(NT, NT == kWave ? 1 : 4) void sums_kernel(VerifyTruncatedArgs a) {
    __shared__ law::Smem<NT> sm;
    const int r = blockIdx.x / kParts, part = blockIdx.x % kParts;
    const Span s = span(a, r);
    const Decision o = decide(a, r, s);  // every wave for itself
    if (o.fault) return;
    const Drawn<DT, NT> drawn(a, r, s, o.L, kParts * NT / kWave);
    const double total = sum_part(drawn, sm, part);
    if (threadIdx.x == 0) a.sums[(int64_t)r * kVerifyParts + part] = total;
}

// Launch 3: outputs and the token at L, a workgroup per request.
template <sv_dtype DT, int NT, int kParts>
__global__ __launch_bounds__(NT, NT == kWave ? 1 : 4) void decide_kernel(VerifyTruncatedArgs a) {
    __shared__ law::Smem<NT> sm;
    const int r = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int k_max = a.k_max;
    const Span s = span(a, r);
    const Decision o = decide(a, r, s);
    int32_t* out = a.out_tokens + (int64_t)r * (k_max + 1);
    if (wave == 0) {
        const int j = lane;
        if (o.fault && lane == 0) raise_error(a.dev_error, o.fault);
        for (int i = j; i <= k_max; i += kWave) {
            if (o.fault) out[i] = -1;
            else if (i != o.L) out[i] = i < o.L ? o.d : -1;
        }
        if (j < k_max) {
            const int64_t at = (int64_t)r * k_max + j;
            if (a.out_p_draft) a.out_p_draft[at] = o.fault || j >= s.b ? -1.0f : (float)o.p;
            if (a.out_q_draft) a.out_q_draft[at] = o.fault || j >= s.b ? -1.0f : (float)o.q;
        }
        if (j == 0) {
            a.out_accepted[r] = o.fault ? -1 : o.L;
            if (a.out_residual_mass && (o.fault || o.L == s.b)) a.out_residual_mass[r] = -1.0f;
        }
    }
    if (o.fault) return;
    Drawn<DT, NT> drawn(a, r, s, o.L, kParts * NT / kWave);
    double sums[kParts], total = 0.0;
#pragma unroll
    for (int i = 0; i < kParts; ++i) sums[i] = a.sums[(int64_t)r * kVerifyParts + i];
#pragma unroll
    for (int i = 0; i < kParts; ++i) total += sums[i];
    if (drawn.minus && threadIdx.x == 0 && a.out_residual_mass)
        a.out_residual_mass[r] = (float)total;
    if (total == 0.0) {  // no residual mass: p itself (rare: summed here)
        drawn.minus = false;
#pragma unroll 1
        for (int i = 0; i < kParts; ++i) {
            const double x = sum_part(drawn, sm, i);
#pragma unroll
            for (int e = 0; e < kParts; ++e) sums[e] = e == i ? x : sums[e];
            total += x;
        }
    }
    // the part that holds the crossing; if rounding leaves none, the last of
    // any weight, and in it the last id of any
    double goal = (double)o.v * total, before = 0.0, at = 0.0;
    int part = -1, positive = 0;
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        if (part < 0 && before + sums[i] > goal) part = i, at = before;
        if (sums[i] > 0.0) positive = i;
        before += sums[i];
    }
    goal = part < 0 ? (double)law::kInf : goal - at;
    if (part < 0) part = positive;
    sum_part(drawn, sm, part);
    const int base = part * (NT / kWave);
    const int tok = law::walk_row(
        sm, sm.redd, NT / kWave, goal, drawn.prow.steps,
        [&](int g, int st, int l) { return drawn.prow.first_id(base + g, st, l); }, a.vocab,
        [&](int id0, double* x) { drawn.of8(id0, x); });
    if (threadIdx.x == 0) out[o.L] = tok;
}

template <sv_dtype DT>
hipError_t run(const VerifyTruncatedArgs& a, hipStream_t stream) {
    const unsigned slots = (unsigned)a.n_req * (2 * a.k_max + 1);
    // two workgroups of 512 threads share a CU in the first launch, whose rows
    // are many; rows of fewer than 8 ids take one wave
    if (a.vocab < 8) laws_kernel<DT, kWave><<<slots, kWave, 0, stream>>>(a);
    else laws_kernel<DT, 512><<<slots, 512, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.vocab < 8) {
        sums_kernel<DT, kWave, 1><<<a.n_req, kWave, 0, stream>>>(a);
        decide_kernel<DT, kWave, 1><<<a.n_req, kWave, 0, stream>>>(a);
    } else {
        constexpr int P = kVerifyParts;
        sums_kernel<DT, 512, P><<<a.n_req * P, 512, 0, stream>>>(a);
        decide_kernel<DT, 512, P><<<a.n_req, 512, 0, stream>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_verify_truncated(const VerifyTruncatedArgs& a, hipStream_t stream) {
    return a.dtype == SV_BF16 ? run<SV_BF16>(a, stream) : run<SV_F32>(a, stream);
}

}  // namespace sv
