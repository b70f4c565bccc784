// sv_verify_truncated: verification of the kept rows under truncated laws
// (temperature, top-k, top-p, min-p of each request; sv_law.h).  The rule is
// sv_verify's (rejection sampling keeps the target's law), with p and q the
// truncated laws.
//
// Launch 1, one 512-thread workgroup per row slot: the law of each target row
// 0 .. b and draft row 0 .. b - 1 of a request (LawRecord), and the weight it
// gives the position's draft id.  Launch 2, one workgroup per request: wave 0
// decides (lane j: position j), then the token at L is drawn over the one or
// two rows that decide it, in 64 bits: each wave sums a contiguous segment of
// ids, the wave that holds the crossing walks its segment again.
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
    const law::Result res = law::find_law(row, set, sm);
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

struct DecideSmem {
    int L, fault;
    float v;
};

template <sv_dtype DT, int kDecide>
__global__ __launch_bounds__(kDecide, kDecide == kWave ? 1 : 4) void decide_kernel(VerifyTruncatedArgs a) {
    using Row = law::Row<DT, kDecide>;
    __shared__ law::Smem<kDecide> sm;
    __shared__ DecideSmem ds;
    const int r = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int k_max = a.k_max;
    const Span s = span(a, r);
    const LawRecord* laws = a.laws + (int64_t)r * (2 * k_max + 1);
    const law::Settings pset = law::settings(a.target_law, r, a.vocab);
    const law::Settings qset = law::settings(a.draft_law, r, a.vocab);
    int32_t* out = a.out_tokens + (int64_t)r * (k_max + 1);
    if (wave == 0) {
        const int j = lane;
        int fault = s.ok ? 0 : SV_DEV_BAD_CU_ROWS;
        // settings of the draft's law matter only where a draft row is read
        if (pset.bad || (qset.bad && s.ok && s.b > 0)) fault |= SV_DEV_BAD_PARAM;
        float u = 0.0f, v = 0.0f;
        draw_uniforms(a.seed, a.step, (uint32_t)r, (uint32_t)j, &u, &v);
        bool acc = true;
        double p = -1.0, q = -1.0;
        int d = -1;
        if (s.ok) {
            if (j < s.b) {
                d = a.draft_tokens[(int64_t)r * k_max + j];
                if (d < 0 || d >= a.vocab) fault |= SV_DEV_BAD_TOKEN;
                const LawRecord t = laws[j], w = laws[k_max + 1 + j];
                fault |= t.fault | w.fault;
                if (!(t.fault | w.fault)) {
                    p = t.drafted / t.total;
                    q = w.drafted / w.total;
                    acc = q > 0.0 ? (double)u < p / q : p > 0.0;
                }
            }
            if (j == 0) fault |= laws[s.b].fault;
        }
        fault = wave_or_int(fault);
        const uint64_t rej = __ballot(!acc);
        const int L = rej ? __builtin_ctzll(rej) : s.b;
        if (lane == 0) {
            ds.L = L;
            ds.fault = fault;
        }
        if (j == L) ds.v = v;
        if (L == kWave && lane == 0) {
            float u2;
            draw_uniforms(a.seed, a.step, (uint32_t)r, (uint32_t)L, &u2, &v);
            ds.v = v;
        }
        if (fault && lane == 0) raise_error(a.dev_error, fault);
        for (int i = j; i <= k_max; i += kWave) {
            if (fault) out[i] = -1;
            else if (i != L) out[i] = i < L ? d : -1;
        }
        if (j < k_max) {
            const int64_t o = (int64_t)r * k_max + j;
            if (a.out_p_draft) a.out_p_draft[o] = fault || j >= s.b ? -1.0f : (float)p;
            if (a.out_q_draft) a.out_q_draft[o] = fault || j >= s.b ? -1.0f : (float)q;
        }
        if (j == 0) {
            a.out_accepted[r] = fault ? -1 : L;
            if (a.out_residual_mass && (fault || L == s.b)) a.out_residual_mass[r] = -1.0f;
        }
    }
    __syncthreads();
    if (ds.fault) return;
    const int L = ds.L;
    const bool residual = L < s.b;
    const LawRecord pr = laws[L];
    const law::Weigher pw = weigher(pr, pset);
    const Row prow(target_row<DT>(a, s.lo, L), a.vocab);
    const double ip = 1.0 / pr.total;
    law::Weigher qw = pw;
    Row qrow = prow;
    double iq = 0.0;
    if (residual) {
        const LawRecord qr = laws[k_max + 1 + L];
        qw = weigher(qr, qset);
        qrow = Row(draft_row<DT>(a, r, L), a.vocab);
        iq = 1.0 / qr.total;
    }
    bool minus = residual;
    const auto weights = [&](int id0, double* x) {
        float z[8], y[8];
        prow.load(id0, z);
        if (minus) qrow.load(id0, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = pw(z[e], id0 + e);
            if (minus && x[e] > 0.0) x[e] = fmax(0.0, x[e] * ip - qw(y[e], id0 + e) * iq);
        }
    };
    // only ids of p's support weigh anything, in the residual too
    const auto sum_row = [&]() {
        double part = 0.0;
        law::compact(prow, sm, [&](float z) { return z >= pw.zc && z > -law::kInf; },
                     [&](float z, int id) {
                         double x = pw(z, id);
                         if (minus) x = fmax(0.0, x * ip - qw(qrow.one(id), id) * iq);
                         part += x;
                     });
        return law::block_sum(part, sm);
    };
    double total = sum_row();
    if (residual && threadIdx.x == 0 && a.out_residual_mass)
        a.out_residual_mass[r] = (float)total;
    if (total == 0.0) {  // no residual mass: p itself
        minus = false;
        total = sum_row();
    }
    const int tok = law::walk_row(
        sm, (double)ds.v * total, prow.steps,
        [&](int w, int st, int l) { return prow.first_id(w, st, l); }, a.vocab, weights);
    if (threadIdx.x == 0) out[L] = tok;
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
    if (a.vocab < 8) decide_kernel<DT, kWave><<<a.n_req, kWave, 0, stream>>>(a);
    else decide_kernel<DT, 1024><<<a.n_req, 1024, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_verify_truncated(const VerifyTruncatedArgs& a, hipStream_t stream) {
    return a.dtype == SV_BF16 ? run<SV_BF16>(a, stream) : run<SV_F32>(a, stream);
}

}  // namespace sv
