// What requests have said, and the logits adjusted for it (gfx950, wave64):
// sv_history_clear, sv_history_add, sv_adjust_logits.
#include "sv_device.h"
#include "sv_launch.h"
#include "sv_logits.h"

namespace sv {
namespace {

constexpr float kInf = __builtin_inff();

// ------------------------------------------------------------------ history

// One workgroup a slot: the listed counts, or all of them where the list did
// not hold every id.
__global__ __launch_bounds__(1024) void clear_kernel(sv_history h, const int32_t* slots,
                                                     int32_t* dev_error) {
    const int slot = slots != nullptr ? slots[blockIdx.x] : (int)blockIdx.x;
    if (slot < 0 || slot >= h.n_slots) {
        if (threadIdx.x == 0) raise_error(dev_error, SV_DEV_BAD_SLOT);
        return;
    }
    const int n = h.n_seen[slot];
    int32_t* counts = h.counts + (int64_t)slot * h.vocab;
    if (n <= h.cap) {
        const int32_t* seen = h.seen + (int64_t)slot * h.cap;
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            const int x = seen[i];
            if (x >= 0 && x < h.vocab) counts[x] = 0;
        }
    } else {
        for (int x = threadIdx.x; x < h.vocab; x += blockDim.x) counts[x] = 0;
    }
    __syncthreads();
    if (threadIdx.x == 0) h.n_seen[slot] = 0;
}

// One thread an id.  The count's old value tells the one thread that listed ids
// new to the slot belong to; a wave takes their places in the list with one add.
__global__ __launch_bounds__(256) void add_kernel(HistoryAddArgs a, int blocks_a_row) {
    const sv_history& h = a.history;
    const int row = blockIdx.x / blocks_a_row;
    const int i = (blockIdx.x - row * blocks_a_row) * 256 + threadIdx.x;
    const int slot = a.slots != nullptr ? a.slots[row] : row;
    if (slot < 0 || slot >= h.n_slots) {
        if (threadIdx.x == 0) raise_error(a.dev_error, SV_DEV_BAD_SLOT);
        return;
    }
    const int x = i < a.width ? a.tokens[(int64_t)row * a.tokens_ld + i] : -1;
    bool fresh = false;
    if (x >= 0 && x < h.vocab) {
        int32_t* at = h.counts + (int64_t)slot * h.vocab + x;
        fresh = (a.in_prompt ? atomicOr(at, 1) : atomicAdd(at, 2)) == 0;
    } else if (x != -1) {
        raise_error(a.dev_error, SV_DEV_BAD_TOKEN);
    }
    const uint64_t who = __ballot(fresh);
    if (who == 0) return;
    const int lane = threadIdx.x & 63, first = __ffsll((unsigned long long)who) - 1;
    int base = 0;
    if (lane == first) base = atomicAdd(h.n_seen + slot, __popcll(who));
    base = __shfl(base, first) + __popcll(who & ((1ull << lane) - 1));
    if (fresh && base < h.cap) h.seen[(int64_t)slot * h.cap + base] = x;
}

// ------------------------------------------------------------------- adjust
//
// One workgroup takes part of a row.  First every id of the part is copied with
// the mask applied, 16 bytes a thread (in place only the masked vectors are
// written); then the few ids that the request has said, drafted or biased are
// computed from the row's own logits and written over.  Each of those ids is
// one thread's: listed ids by their place in the list, drafted ones that are
// not listed by their first occurrence, biased ones if they are neither.

template <typename T>
struct Row;
template <>
struct Row<float> {
    static constexpr int kVec = 4;
    static __device__ __forceinline__ float get(const void* row, int x) {
        return static_cast<const float*>(row)[x];
    }
    static __device__ __forceinline__ void put(void* row, int x, float v) {
        static_cast<float*>(row)[x] = v;
    }
    // -inf where the bit of `allowed` is 0
    static __device__ __forceinline__ void mask(uint32_t (&w)[4], uint32_t allowed) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (allowed >> i) & 1 ? w[i] : 0xff800000u;
    }
};
template <>
struct Row<uint16_t> {
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float get(const void* row, int x) {
        return __uint_as_float((uint32_t)static_cast<const uint16_t*>(row)[x] << 16);
    }
    static __device__ __forceinline__ void put(void* row, int x, float v) {
        const __bf16 b = (__bf16)v;  // to the nearest, ties to even
        static_cast<__bf16*>(row)[x] = b;
    }
    static __device__ __forceinline__ void mask(uint32_t (&w)[4], uint32_t allowed) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = (allowed >> (2 * i)) & 1 ? w[i] : 0xff80u;
            const uint32_t hi = (allowed >> (2 * i + 1)) & 1 ? w[i] : 0xff800000u;
            w[i] = (lo & 0xffffu) | (hi & 0xffff0000u);
        }
    }
};

constexpr int kAdjustThreads = 256;

template <typename T>
__global__ __launch_bounds__(kAdjustThreads) void adjust_kernel(AdjustArgs a) {
    constexpr int kVec = Row<T>::kVec;
    __shared__ int drafts[SV_MAX_DRAFT];
    const int tid = threadIdx.x;
    const int row = blockIdx.x / a.parts, part = blockIdx.x - row * a.parts;
    const int begin = part * a.part_len, end = min(a.vocab, begin + a.part_len);
    const char* in = static_cast<const char*>(a.logits) + (int64_t)row * a.ld * sizeof(T);
    char* out = static_cast<char*>(a.out) + (int64_t)row * a.out_ld * sizeof(T);
    const bool in_place = a.logits == a.out;

    const int r = a.row_req != nullptr ? a.row_req[row] : row;
    if (r == -1) return;
    const int j = a.row_pos != nullptr ? a.row_pos[row] : 0;
    int fault =
        r < 0 || r >= a.n_req || j < 0 || (a.penalised && j > a.k_max) ? SV_DEV_BAD_CU_ROWS : 0;
    float rho = 1.0f, phi = 0.0f, pi = 0.0f;
    int slot = 0, n_seen = 0, b0 = 0, b1 = 0;
    const uint32_t* mask = nullptr;
    const bool known = fault == 0;
    const bool said = a.penalised && a.history.counts != nullptr;
    if (known) {
        if (said) {
            slot = a.slots != nullptr ? a.slots[r] : r;
            if (slot < 0 || slot >= a.history.n_slots) {
                fault |= SV_DEV_BAD_SLOT;
                slot = 0;
            } else {
                n_seen = a.history.n_seen[slot];
            }
        }
        if (a.penalised) {
            const sv_penalties& p = a.penalties;
            if (p.repetition != nullptr) rho = p.repetition[r];
            if (p.frequency != nullptr) phi = p.frequency[r];
            if (p.presence != nullptr) pi = p.presence[r];
            if (!is_finite_bits(rho) || !(rho > 0.0f) || !is_finite_bits(phi) ||
                !is_finite_bits(pi))
                fault |= SV_DEV_BAD_PARAM;
            if (tid < j) {
                const int d = a.draft_tokens[(int64_t)r * a.k_max + tid];
                drafts[tid] = d;
                if (d < 0 || d >= a.vocab) fault |= SV_DEV_BAD_TOKEN;
            }
        }
        if (a.bias.n_entries > 0) {
            b0 = a.bias.start[r];
            b1 = a.bias.start[r + 1];
            if (b0 < 0 || b1 < b0 || b1 > a.bias.n_entries) {
                fault |= SV_DEV_BAD_PARAM;
                b0 = b1 = 0;
            }
            for (int i = b0 + tid; i < b1; i += kAdjustThreads) {
                const int x = a.bias.ids[i];
                if (x < 0 || x >= a.vocab || (i > b0 && a.bias.ids[i - 1] >= x))
                    fault |= SV_DEV_BAD_TOKEN;
                const float v = a.bias.values[i];
                if (!is_finite_bits(v) && __float_as_uint(v) != 0xff800000u)
                    fault |= SV_DEV_BAD_PARAM;
            }
        }
        if (a.masked) {
            const int m = a.mask.row_mask != nullptr ? a.mask.row_mask[row] : row;
            if (m < -1 || m >= a.mask.n_masks) fault |= SV_DEV_BAD_PARAM;
            else if (m >= 0)
                mask = reinterpret_cast<const uint32_t*>(a.mask.bits) + (int64_t)m * a.mask.ld;
        }
    }
    if (__syncthreads_or(fault)) {
        raise_error(a.dev_error, fault);
        for (int x = begin + tid; x < end; x += kAdjustThreads)
            Row<T>::put(out, x, __builtin_nanf(""));
        return;
    }

    // every id of the part; vectors start at multiples of kVec ids, so that a
    // vector's bits lie in one word
    if (!in_place || mask != nullptr) {
        const int full = begin + (end - begin) / kVec * kVec;
        for (int x = begin + tid * kVec; x < full; x += kAdjustThreads * kVec) {
            uint32_t allowed = ~0u;
            if (mask != nullptr) allowed = mask[x >> 5] >> (x & 31);
            constexpr uint32_t kAll = (1u << kVec) - 1;
            if (in_place && (allowed & kAll) == kAll) continue;
            uint32_t w[4] = {};
            if ((allowed & kAll) != 0) __builtin_memcpy(w, in + (int64_t)x * sizeof(T), 16);
            if (mask != nullptr) Row<T>::mask(w, allowed);
            __builtin_memcpy(out + (int64_t)x * sizeof(T), w, 16);
        }
        const int x = full + tid;
        if (x < end) {
            const bool ok = mask == nullptr || ((mask[x >> 5] >> (x & 31)) & 1);
            Row<T>::put(out, x, ok ? Row<T>::get(in, x) : -kInf);
        }
    }
    if (!a.penalised && b0 == b1) return;
    __syncthreads();

    const int32_t* counts =
        said ? a.history.counts + (int64_t)slot * a.history.vocab : nullptr;
    const int n_drafts = a.penalised ? j : 0;
    // ids of this part that the mask allows
    auto mine = [&](int x) {
        return x >= begin && x < end && (mask == nullptr || ((mask[x >> 5] >> (x & 31)) & 1));
    };
    auto drafted = [&](int x, int before) {
        int n = 0;
        for (int i = 0; i < before; ++i) n += drafts[i] == x;
        return n;
    };
    // z3 of an id that history holds (twice the times it was emitted, + 1) and the
    // drafts repeat
    auto adjust = [&](int x, int held, int again) {
        float z = Row<T>::get(in, x);
        z = z > 0.0f ? __fdiv_rn(z, rho) : z * rho;
        const int c = (held >> 1) + again;
        if (c > 0) z = z - phi * (float)c - pi;
        int lo = b0, hi = b1;  // the first entry not below x
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (a.bias.ids[mid] < x) lo = mid + 1;
            else hi = mid;
        }
        if (lo < b1 && a.bias.ids[lo] == x) z += a.bias.values[lo];
        Row<T>::put(out, x, z);
    };
    if (said) {
        if (n_seen <= a.history.cap) {
            const int32_t* seen = a.history.seen + (int64_t)slot * a.history.cap;
            for (int i = tid; i < n_seen; i += kAdjustThreads) {
                const int x = seen[i];
                if (mine(x)) adjust(x, counts[x], drafted(x, n_drafts));
            }
        } else {
            for (int x = begin + tid; x < end; x += kAdjustThreads) {
                const int held = counts[x];
                if (held != 0 && mine(x)) adjust(x, held, drafted(x, n_drafts));
            }
        }
    }
    if (tid < n_drafts) {
        const int x = drafts[tid];
        if (mine(x) && drafted(x, tid) == 0 && (!said || counts[x] == 0))
            adjust(x, 0, drafted(x, n_drafts));
    }
    for (int i = b0 + tid; i < b1; i += kAdjustThreads) {
        const int x = a.bias.ids[i];
        if (mine(x) && (!said || counts[x] == 0) && drafted(x, n_drafts) == 0)
            Row<T>::put(out, x, Row<T>::get(in, x) + a.bias.values[i]);
    }
}

}  // namespace

hipError_t launch_history_clear(const sv_history& h, const int32_t* slots, int n,
                                int32_t* dev_error, hipStream_t stream) {
    clear_kernel<<<(unsigned)n, 1024, 0, stream>>>(h, slots, dev_error);
    return hipGetLastError();
}

hipError_t launch_history_add(const HistoryAddArgs& a, hipStream_t stream) {
    const int blocks = (a.width + 255) / 256;
    add_kernel<<<(unsigned)(a.n * blocks), 256, 0, stream>>>(a, blocks);
    return hipGetLastError();
}

hipError_t launch_adjust(const AdjustArgs& a, hipStream_t stream) {
    const unsigned grid = (unsigned)((int64_t)a.n_rows * a.parts);
    if (a.dtype == SV_BF16)
        adjust_kernel<uint16_t><<<grid, kAdjustThreads, 0, stream>>>(a);
    else
        adjust_kernel<float><<<grid, kAdjustThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace sv
