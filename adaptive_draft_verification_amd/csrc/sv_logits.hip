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

// PER ids a thread.  The count's old value tells the one thread that listed ids new to
// the slot belong to; a wave takes their places in the list with one add.  Bound by the
// atomics' way to the counts' lines, all over memory, and by the adds to a row's one
// n_seen: with 4 ids in flight a thread 256 x 4096 ids of 129,280 take 35 us (45 one at a
// time), few ids their launch.
template <int PER>
__global__ __launch_bounds__(256) void add_kernel(HistoryAddArgs a, int blocks_a_row) {
    const sv_history& h = a.history;
    const int row = blockIdx.x / blocks_a_row;
    const int i0 = (blockIdx.x - row * blocks_a_row) * 256 * PER + threadIdx.x;
    const int slot = a.slots != nullptr ? a.slots[row] : row;
    if (slot < 0 || slot >= h.n_slots) {
        if (threadIdx.x == 0) raise_error(a.dev_error, SV_DEV_BAD_SLOT);
        return;
    }
    const int32_t* tokens = a.tokens + (int64_t)row * a.tokens_ld;
    int x[PER], was[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) x[j] = i0 + j * 256 < a.width ? tokens[i0 + j * 256] : -1;
    bool wrong = false;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        was[j] = 1;
        if (x[j] >= 0 && x[j] < h.vocab) {
            int32_t* at = h.counts + (int64_t)slot * h.vocab + x[j];
            was[j] = a.in_prompt ? atomicOr(at, 1) : atomicAdd(at, 2);
        } else if (x[j] != -1) {
            wrong = true;
        }
    }
    if (wrong) raise_error(a.dev_error, SV_DEV_BAD_TOKEN);
    const int lane = threadIdx.x & 63;
    int before[PER], all = 0;  // ids of the wave that come first in the list
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const uint64_t who = __ballot(was[j] == 0);
        before[j] = all + __popcll(who & ((1ull << lane) - 1));
        all += __popcll(who);
    }
    if (all == 0) return;
    int base = 0;
    if (lane == 0) base = atomicAdd(h.n_seen + slot, all);
    base = __shfl(base, 0);
#pragma unroll
    for (int j = 0; j < PER; ++j)
        if (was[j] == 0 && base + before[j] < h.cap)
            h.seen[(int64_t)slot * h.cap + base + before[j]] = x[j];
}

// ------------------------------------------------------------------- adjust
//
// Bound by the rows, read and written once: 256 x 1 .. 8 rows of 129,280 bf16 with
// penalties, biases and masks 156 us (4.0 TB/s; the rows alone copied 114), in place 105,
// fp32 269 (231) and 163, 1 row of 128,255 fp32 5.4.  That is with 2560 ids said by each
// request, whose list every workgroup of its rows reads; with 274 of them 123 and 43, with
// 14,200 324 and 253.  One workgroup takes a part of a row.
// Out of place (kStaged) the part goes through LDS: the few ids that the request
// has said, drafted or biased are adjusted there, and the part leaves with the mask
// applied.  In place only the masked vectors and those few ids are touched.  Each of
// the ids is one thread's, which finds its count and its bias itself.
// A part is every parts-th tile of kAdjustTile ids: the ids that texts repeat most
// are neighbours (the lowest ones, as tokenisers number them), and would be one
// workgroup's otherwise.

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
constexpr int kPlaces = 6;  // places a thread looks at, their loads in flight together

template <typename T, bool kStaged>
__global__ __launch_bounds__(kAdjustThreads, kStaged ? 4 : 8) void adjust_kernel(AdjustArgs a) {
    constexpr int kVec = Row<T>::kVec;
    constexpr int kVecs = kAdjustPartBytes / 16 / kAdjustThreads;  // a thread's, staged
    __shared__ uint4 staged[kStaged ? kAdjustPartBytes / 16 : 1];
    __shared__ int drafts[SV_MAX_DRAFT];
    // bit x % kSieve: x may be drafted or biased (a bias is found by halving the
    // list, some steps of memory latency: not for every id that was said)
    constexpr int kSieve = 8192;
    __shared__ uint32_t sieve[kSieve / 32];
    __shared__ int found[kPlaces * kAdjustThreads], n_found;
    const int tid = threadIdx.x;
    const int row = blockIdx.x / a.parts, part = blockIdx.x - row * a.parts;
    const char* in = static_cast<const char*>(a.logits) + (int64_t)row * a.ld * sizeof(T);
    char* out = static_cast<char*>(a.out) + (int64_t)row * a.out_ld * sizeof(T);
    // ids of the part: whole tiles, and what the last one lacks; parts is a power of
    // two
    const int tiles = (a.vocab + kAdjustTile - 1) / kAdjustTile;
    const int my_tiles = part < tiles ? (tiles - part + a.parts - 1) / a.parts : 0;
    const bool has_last = my_tiles > 0 && ((tiles - 1) & (a.parts - 1)) == part;
    const int my_ids = my_tiles * kAdjustTile - (has_last ? tiles * kAdjustTile - a.vocab : 0);
    const int vecs = my_ids / kVec;
    auto id_at = [&](int i) {
        return ((i / kAdjustTile) * a.parts + part) * kAdjustTile + i % kAdjustTile;
    };
    auto mine = [&](int x) {
        return x >= 0 && x < a.vocab && ((x / kAdjustTile) & (a.parts - 1)) == part;
    };

    const int r = a.row_req != nullptr ? a.row_req[row] : row;
    if (r == -1) return;
    // the steps from here to the counts wait for memory five times, one for the
    // other: the part is on its way meanwhile
    uint32_t w[kVecs][4];
    if constexpr (kStaged) {
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            const int v = u * kAdjustThreads + tid;
            if (v < vecs) __builtin_memcpy(w[u], in + (int64_t)id_at(v * kVec) * sizeof(T), 16);
        }
    }
    for (int i = tid; i < kSieve / 32; i += kAdjustThreads) sieve[i] = 0;
    if (tid == 0) n_found = 0;
    __syncthreads();
    auto sift = [&](int x) { atomicOr(&sieve[(x % kSieve) / 32], 1u << (x % 32)); };
    const int j = a.row_pos != nullptr ? a.row_pos[row] : 0;
    int fault =
        r < 0 || r >= a.n_req || j < 0 || (a.penalised && j > a.k_max) ? SV_DEV_BAD_CU_ROWS : 0;
    float rho = 1.0f, phi = 0.0f, pi = 0.0f;
    int slot = 0, n_seen = 0, b0 = 0, b1 = 0;
    const uint32_t* mask = nullptr;
    const bool said = a.penalised && a.history.counts != nullptr;
    const int n_drafts = a.penalised && fault == 0 ? j : 0;
    if (fault == 0) {
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
            if (tid < n_drafts) {
                const int d = a.draft_tokens[(int64_t)r * a.k_max + tid];
                drafts[tid] = d;
                if (d < 0 || d >= a.vocab) fault |= SV_DEV_BAD_TOKEN;
                else sift(d);
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
                else sift(x);
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
    if constexpr (kStaged) {
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            const int v = u * kAdjustThreads + tid;
            if (v < vecs) staged[v] = make_uint4(w[u][0], w[u][1], w[u][2], w[u][3]);
        }
        const int i = vecs * kVec + tid;
        if (i < my_ids) Row<T>::put(staged, i, Row<T>::get(in, id_at(i)));
    }
    if (__syncthreads_or(fault)) {
        raise_error(a.dev_error, fault);
        for (int i = tid; i < my_ids; i += kAdjustThreads)
            Row<T>::put(out, id_at(i), __builtin_nanf(""));
        return;
    }
    auto allowed = [&](int x) { return mask == nullptr || ((mask[x >> 5] >> (x & 31)) & 1); };

    // in place: vectors with an id that the mask does not allow; vectors start at
    // multiples of kVec ids, so that a vector's bits lie in one word
    constexpr uint32_t kAll = (1u << kVec) - 1;
    if (!kStaged && mask != nullptr) {
        for (int v = tid; v < vecs; v += kAdjustThreads) {
            const int x = id_at(v * kVec);
            const uint32_t bits = (mask[x >> 5] >> (x & 31)) & kAll;
            if (bits == kAll) continue;
            uint32_t t[4] = {};
            if (bits != 0) __builtin_memcpy(t, in + (int64_t)x * sizeof(T), 16);
            Row<T>::mask(t, bits);
            __builtin_memcpy(out + (int64_t)x * sizeof(T), t, 16);
        }
        const int i = vecs * kVec + tid;
        if (i < my_ids && !allowed(id_at(i))) Row<T>::put(out, id_at(i), -kInf);
        __syncthreads();
    }

    // Ids stand in the history's list (or among its counts of the part, where the
    // list did not hold every id); biases and drafts are looked at where they are
    // not in the history, equal drafts at the first.
    const int32_t* counts =
        said ? a.history.counts + (int64_t)slot * a.history.vocab : nullptr;
    const bool list = n_seen <= a.history.cap;
    const int n_said = !said ? 0 : list ? n_seen : my_ids;
    const int n_bias = b1 - b0;
    auto bias_of = [&](int x) {  // x's entry, or -1
        int lo = b0, hi = b1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (a.bias.ids[mid] < x) lo = mid + 1;
            else hi = mid;
        }
        return lo < b1 && a.bias.ids[lo] == x ? lo : -1;
    };
    auto sifted = [&](int x) { return (sieve[(x % kSieve) / 32] >> (x % 32)) & 1; };
    // z3 of x, with its entry (-1: it has none, -2: to be looked for)
    auto adjust = [&](int x, int held, int entry) {
        if (sifted(x)) {
            for (int e = 0; e < n_drafts; ++e) held += drafts[e] == x ? 2 : 0;
            if (entry == -2) entry = bias_of(x);
        }
        void* row_at = kStaged ? static_cast<void*>(staged) : out;
        const int i = kStaged ? x / (kAdjustTile * a.parts) * kAdjustTile + x % kAdjustTile : x;
        float z = Row<T>::get(row_at, i);
        if (held > 0) z = z > 0.0f ? __fdiv_rn(z, rho) : z * rho;
        if (held > 1) z = z - phi * (float)(held >> 1) - pi;
        if (entry >= 0) z += a.bias.values[entry];
        Row<T>::put(row_at, i, z);
    };
    for (int from = 0; from < n_said; from += kPlaces * kAdjustThreads) {
        // the part's ids among the next places, packed: one in parts of a list's
        if (from > 0) {
            __syncthreads();
            if (tid == 0) n_found = 0;
            __syncthreads();
        }
        int x[kPlaces];
#pragma unroll
        for (int u = 0; u < kPlaces; ++u) {
            const int i = from + u * kAdjustThreads + tid;
            x[u] = -1;
            if (i < n_said)
                x[u] = list ? a.history.seen[(int64_t)slot * a.history.cap + i] : id_at(i);
        }
#pragma unroll
        for (int u = 0; u < kPlaces; ++u)
            if (mine(x[u])) found[atomicAdd(&n_found, 1)] = x[u];
        __syncthreads();
        for (int i = tid; i < n_found; i += kAdjustThreads) {
            const int y = found[i], held = counts[y];
            // staged parts are masked as they leave
            if (held != 0 && (kStaged || allowed(y))) adjust(y, held, -2);
        }
    }
    for (int i = tid; i < n_bias + n_drafts; i += kAdjustThreads) {
        const int d = i - n_bias;  // below 0: a bias
        const int x = d < 0 ? a.bias.ids[b0 + i] : drafts[d];
        if (!mine(x) || !(kStaged || allowed(x)) || (said && counts[x] != 0)) continue;
        bool again = d >= 0 && bias_of(x) >= 0;
        for (int e = 0; e < d; ++e) again |= drafts[e] == x;
        if (!again) adjust(x, 0, d < 0 ? b0 + i : -1);
    }
    if constexpr (kStaged) {
        __syncthreads();
        for (int v = tid; v < vecs; v += kAdjustThreads) {
            const int x = id_at(v * kVec);
            const uint4 s = staged[v];
            uint32_t t[4] = {s.x, s.y, s.z, s.w};
            if (mask != nullptr) Row<T>::mask(t, mask[x >> 5] >> (x & 31));
            __builtin_memcpy(out + (int64_t)x * sizeof(T), t, 16);
        }
        const int i = vecs * kVec + tid;
        if (i < my_ids) {
            const int x = id_at(i);
            Row<T>::put(out, x, allowed(x) ? Row<T>::get(staged, i) : -kInf);
        }
    }
}

template <typename T>
void run_adjust(const AdjustArgs& a, hipStream_t stream) {
    const unsigned grid = (unsigned)((int64_t)a.n_rows * a.parts);
    if (a.logits == a.out)
        adjust_kernel<T, false><<<grid, kAdjustThreads, 0, stream>>>(a);
    else
        adjust_kernel<T, true><<<grid, kAdjustThreads, 0, stream>>>(a);
}

}  // namespace

hipError_t launch_history_clear(const sv_history& h, const int32_t* slots, int n,
                                int32_t* dev_error, hipStream_t stream) {
    clear_kernel<<<(unsigned)n, 1024, 0, stream>>>(h, slots, dev_error);
    return hipGetLastError();
}

hipError_t launch_history_add(const HistoryAddArgs& a, hipStream_t stream) {
    // four a thread where that leaves a workgroup for half of the CUs
    if ((int64_t)a.n * a.width >= 128 * 1024 && a.width > 256) {
        const int blocks = (int)(((int64_t)a.width + 1023) / 1024);
        add_kernel<4><<<(unsigned)(a.n * blocks), 256, 0, stream>>>(a, blocks);
    } else {
        const int blocks = (a.width + 255) / 256;
        add_kernel<1><<<(unsigned)(a.n * blocks), 256, 0, stream>>>(a, blocks);
    }
    return hipGetLastError();
}

hipError_t launch_adjust(const AdjustArgs& a, hipStream_t stream) {
    if (a.dtype == SV_BF16) run_adjust<uint16_t>(a, stream);
    else run_adjust<float>(a, stream);
    return hipGetLastError();
}

}  // namespace sv
