// The paged key-value cache of the packed verify batch (gfx950, wave64):
// sv_cache_append writes a step's new keys and values behind each request's
// context, sv_cache_attend lets the packed rows attend to it.
#include "sv_attend_kernel.h"
#include "sv_device.h"
#include "sv_launch.h"
#include "sv_serve.h"

namespace sv {
namespace {

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
    const float* scales = is_v ? c.v_scale : c.k_scale;
    const float s = scales != nullptr ? scales[h] : 1.0f;
    *reinterpret_cast<int2*>(static_cast<uint8_t*>(is_v ? c.v : c.k) + at) = e4m3_of(w, s);
}

// ------------------------------------------------------------------- attend

// Merges the parts of a (row, head): W waves, wave w the parts w, w + W, ..., lanes
// over the dims; the waves' sums meet in LDS, in a fixed order.  hipcc puts a part's load
// behind the test that ends the sum, so that a wave has one on its way at a time.  A
// request of one part wrote its outputs itself.
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
    // up to 16 parts are one wave's
    if (a.parts <= 16) {
        const int64_t grid = (total + 3) / 4;
        join_kernel<D, F8, 1><<<(unsigned)(grid < 4096 ? grid : 4096), 256, 0, stream>>>(a);
    } else {
        join_kernel<D, F8, 4><<<(unsigned)(total < 4096 ? total : 4096), 256, 0, stream>>>(a);
    }
}

template <int D, bool F8, int MT, bool PG16>
__global__ __launch_bounds__(256, (Attend<D, F8, MT, PG16>::kOccupancy))
void attend_kernel(AttendArgs a) {
    constexpr bool OWN = false;
    const unsigned block = blockIdx.x, blocks = gridDim.x;
    __shared__ typename Attend<D, F8, MT, PG16>::Smem sm;
#include "sv_attend_body.h"
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
