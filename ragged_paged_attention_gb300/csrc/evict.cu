// Eviction of cached keys by their weights (rpa_evict_kv_cache), for sm_103a: a kernel that selects, a block for every
// sequence and KV head, and one that moves.
//
// Of a head's n keys the `keep` of the largest weights stay (the first `sinks` and last `recent` before all others; equal
// weights by lower slot).  Slots below `keep` whose key goes are holes, kept keys behind it movers: as many of one as
// of the other, and the i-th hole takes the i-th mover.  So nothing that is read is written, in place or not, and only the rows
// that have to move do: 2 row_bytes keep (1 - keep / n) for weights in any order.
//
// Selection: weights as integers of their order, the keep-th largest found 11 bits at a time from histograms in
// shared memory, then one pass that counts and one that places, each thread on a run of consecutive slots.
//
// 48 sequences of 4000 to 12000 keys cut to 2048, 8 heads of 128 in bf16: selection 59 us (384 blocks, one an SM: 53
// registers by 1024 threads; latencies of shared memory and barriers over five passes), moving 104 us (0.57 GB, rows of 512 bytes read and written
// all over the pages: 5.4 TB/s), 155 us together.
//
// With positions (kernels of their own, so that calls without are as they were) a key's age is its number, not its slot: the
// numbers of new keys go on behind the greatest in a head, each kept key takes its number along, and the `recent`
// greatest come before all other keys. The slots left behind are as if never used: number -1, weight 0.
// The batch above takes 188 us so (4 bytes more a key read, 8 a key that goes written, no two of them adjacent); a sequence of 3001 keys cut to
// 1024 23 us, 20 without.
#include "common.cuh"
#include "kernels.h"
#include "profile.h"

namespace rpa {

constexpr int kEvictThreads = 1024;  // (48 sequences cut to 2048 keys: 156 us, with 512 threads 162; one 20 and 22)
constexpr int kEvictBins = 2048;
constexpr int kEvictAhead = 8;
constexpr int kEvictHeld = 49152;      // most keys whose order a block holds in shared memory

// Weights as integers of the same order: NaN below all, either zero alike; a kept key above all.
__device__ __forceinline__ uint32_t evict_order(float w) {
    if (w != w) return 0;
    const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Where sequence s's slot i is: its page and the slot in it.
struct EvictSlot {
    size_t page;
    int in_page;
};
__device__ __forceinline__ EvictSlot evict_slot(const EvictArgs& a, int s, int i) {
    const int p = a.page_shift >= 0 ? i >> a.page_shift : i / a.page_size;
    return {(size_t)a.page_indices[(size_t)s * a.pages_per_seq + p], i - p * a.page_size};
}
__device__ __forceinline__ size_t evict_weight(const EvictArgs& a, const EvictSlot& at, int h) {
    return (at.page * a.num_kv_heads + h) * a.page_size + at.in_page;
}

// How many keys of sequence s stay, and its length; -1 where it is left alone (the error word then says why).
__device__ __forceinline__ int evict_keep(const EvictArgs& a, int s, int& n) {
    const int num = a.num_seqs[0];
    if (num < 0 || num > a.max_num_seqs) {
        if (threadIdx.x == 0) set_error(a.err, RPA_DEV_ERR_NUM_SEQS);
        return -1;
    }
    if (s >= num) return -1;
    n = a.kv_lens[s];
    const int budget = a.budgets[s];
    uint32_t bad = 0;
    if (n < 0 || (n > 0 && (n - 1) / a.page_size >= a.pages_per_seq))
        bad = RPA_DEV_ERR_KV_LEN;
    else if (budget < 0 || budget > a.max_keys)
        bad = RPA_DEV_ERR_BUDGET;
    if (bad) {
        if (threadIdx.x == 0) set_error(a.err, bad);
        return -1;
    }
    return min(n, max(budget, a.sinks + a.recent));
}

// A slot that its key has left.
__device__ __forceinline__ void evict_vacate(const EvictArgs& a, size_t at) {
    a.positions[at] = -1;
    if (a.weights_out) a.weights_out[at] = 0.f;
}
// The number of slot i's key: its own, or, where it has none yet, the one that its place among the new keys gives it.
__device__ __forceinline__ long long evict_number(const EvictArgs& a, size_t at, int i, long long base) {
    const int p = a.positions[at];
    return p < 0 ? base + i : p;
}

template <bool AGED>
__global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(const __grid_constant__ EvictArgs a) {
    extern __shared__ uint32_t held[];  // the keys' order, where they fit
    __shared__ int hist[kEvictBins];
    __shared__ long long scan[40];
    __shared__ int s_bad, s_digit, s_above;
    [[maybe_unused]] __shared__ int s_greatest, s_first_new, s_last_new;
    const int s = blockIdx.x / a.num_kv_heads, h = blockIdx.x % a.num_kv_heads, tid = threadIdx.x;
    pdl_launch_dependents();  // (the moving kernel waits for this grid's end)
    int n = 0, keep = evict_keep(a, s, n);
    // every page of the sequence is one of the cache's, or the sequence is left alone
    if (tid == 0) {
        s_bad = 0;
        if constexpr (AGED) {
            s_greatest = s_last_new = -1;
            s_first_new = INT32_MAX;
        }
    }
    __syncthreads();
    if (keep >= 0) {
        const int pages = cdiv(n, a.page_size);
        bool bad = false;
        for (int i = tid; i < pages; i += kEvictThreads)
            bad |= (unsigned)a.page_indices[(size_t)s * a.pages_per_seq + i] >= (unsigned)a.total_num_pages;
        if (bad) s_bad = 1;
    }
    __syncthreads();
    if (keep >= 0 && s_bad) {
        if (tid == 0) set_error(a.err, RPA_DEV_ERR_PAGE);
        keep = -1;
    }
    if (h == 0 && tid == 0) a.kept[s] = keep;
    auto index = [&](int i) { return evict_weight(a, evict_slot(a, s, i), h); };
    [[maybe_unused]] long long base = 0, newest = 0;  // slot i's number where it is new, and the greatest of all
    if constexpr (AGED) {
        if (keep < 0) return;
        int greatest = -1, first_new = INT32_MAX, last_new = -1;
        for (int i = tid; i < n; i += kEvictThreads) {
            const int p = a.positions[index(i)];
            greatest = max(greatest, p);
            if (p < 0) {
                first_new = min(first_new, i);
                last_new = i;
            }
        }
        greatest = __reduce_max_sync(0xffffffffu, greatest);
        first_new = __reduce_min_sync(0xffffffffu, first_new);
        last_new = __reduce_max_sync(0xffffffffu, last_new);
        if ((tid & 31) == 0) {
            atomicMax(&s_greatest, greatest);
            atomicMin(&s_first_new, first_new);
            atomicMax(&s_last_new, last_new);
        }
        __syncthreads();
        base = (long long)s_greatest + 1 - s_first_new;
        newest = s_last_new >= 0 ? base + s_last_new : s_greatest;
        if (tid == 0) a.bases[s * a.num_kv_heads + h] = base;
        if (keep == 0)
            for (int i = tid; i < n; i += kEvictThreads) evict_vacate(a, index(i));
    }
    if (keep <= 0) return;
    int* out = a.slots_out + ((size_t)s * a.num_kv_heads + h) * a.max_keys;
    if (keep == n) {
        for (int i = tid; i < n; i += kEvictThreads) out[i] = i;
        return;
    }
    auto order_of = [&](int i) -> uint32_t {
        if (i < a.sinks) return 0xffffffffu;
        if constexpr (AGED) {
            const size_t at = index(i);
            return evict_number(a, at, i, base) > newest - a.recent ? 0xffffffffu : evict_order(a.weights[at]);
        }
        if (i >= n - a.recent) return 0xffffffffu;
        return evict_order(a.weights[index(i)]);
    };
    const bool fits = n <= a.held;
    if (fits) {
        // (several keys' page and weight on their way at once)
        for (int i0 = tid; i0 < n; i0 += kEvictAhead * kEvictThreads) {
            uint32_t v[kEvictAhead];
#pragma unroll
            for (int u = 0; u < kEvictAhead; ++u) v[u] = order_of(min(i0 + u * kEvictThreads, n - 1));
#pragma unroll
            for (int u = 0; u < kEvictAhead; ++u)
                if (i0 + u * kEvictThreads < n) held[i0 + u * kEvictThreads] = v[u];
        }
        __syncthreads();
    }
    auto order = [&](int i) { return fits ? held[i] : order_of(i); };
    // the keep-th largest: its bits from the top, with the number of keys above what is known of it
    uint32_t top = 0;
    int above = 0, width = 32;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int bits = pass < 2 ? 11 : 10, shift = width - bits;
        for (int i = tid; i < kEvictBins; i += kEvictThreads) hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kEvictThreads) {
            const uint32_t v = order(i);
            if (pass == 0 || v >> width == top) atomicAdd(&hist[v >> shift & ((1u << bits) - 1)], 1);
        }
        __syncthreads();
        // bins from the greatest down, two a thread: the one where the count passes keep
        constexpr int kPer = kEvictBins / kEvictThreads;
        int c[kPer], sum = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum += c[j] = hist[kEvictBins - 1 - (tid * kPer + j)];
        long long total;
        int before = above + (int)block_exclusive_scan((long long)sum, scan, &total);
        if (before < keep && before + sum >= keep) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                if (before < keep && before + c[j] >= keep) {
                    s_digit = kEvictBins - 1 - (tid * kPer + j);
                    s_above = before;
                }
                before += c[j];
            }
        }
        __syncthreads();
        top = top << bits | (uint32_t)s_digit;
        above = s_above;
        width = shift;
    }
    // keys above `top` stay, and of those equal to it the first keep - above
    // (runs of an odd length: 32 threads' slots lie in 32 banks)
    const int ties = keep - above, per = cdiv(n, kEvictThreads) | 1, i0 = min(n, tid * per), i1 = min(n, i0 + per);
    int equal = 0;
    for (int i = i0; i < i1; ++i) equal += order(i) == top;
    long long total;
    const int equal0 = (int)block_exclusive_scan((long long)equal, scan, &total);
    int e = equal0, holes = 0, movers = 0;
    for (int i = i0; i < i1; ++i) {
        const uint32_t v = order(i);
        const bool stays = v > top || (v == top && e < ties);
        e += v == top;
        holes += !stays && i < keep;
        movers += stays && i >= keep;
    }
    const long long before = block_exclusive_scan(((long long)holes << 32) | movers, scan, &total);
    int hole = (int)(before >> 32), mover = (int)(before & 0xffffffffll);
    int* hole_at = a.holes + ((size_t)s * a.num_kv_heads + h) * a.max_keys;
    e = equal0;
    for (int i = i0; i < min(i1, keep); ++i) {
        const uint32_t v = order(i);
        const bool stays = v > top || (v == top && e < ties);
        e += v == top;
        if (stays)
            out[i] = i;
        else
            hole_at[hole++] = i;
    }
    __syncthreads();  // (the block's own writes: its holes are all there)
    for (int i = max(i0, keep); i < i1; ++i) {
        const uint32_t v = order(i);
        const bool stays = v > top || (v == top && e < ties);
        e += v == top;
        if (stays)
            out[hole_at[mover++]] = i;
        else if constexpr (AGED)
            evict_vacate(a, index(i));  // (nobody reads it any more; the slots of movers: by the thread that moves them)
    }
}

// A warp takes 32 slots of a head: their weights, a lane each, and the rows that come from elsewhere, 16 bytes a lane.
template <bool AGED>
__global__ void __launch_bounds__(kEvictMoveThreads) evict_move_kernel(const __grid_constant__ EvictArgs a, int blocks_per_head) {
    __shared__ const uint4* from[kEvictMoveThreads];
    __shared__ uint4* to[kEvictMoveThreads];
    const int head = blockIdx.x / blocks_per_head, s = head / a.num_kv_heads, h = head % a.num_kv_heads;
    const int block = blockIdx.x % blocks_per_head, lane = threadIdx.x & 31, w0 = threadIdx.x & ~31;
    pdl_wait();
    const int keep = a.kept[s];
    if (keep < 0) return;
    if (a.kv_lens_out && h == 0 && block == 0 && threadIdx.x == 0) a.kv_lens_out[s] = keep;
    const int i = block * kEvictMoveThreads + threadIdx.x;
    if (i - lane >= keep) return;
    const int src = i < keep ? a.slots_out[((size_t)s * a.num_kv_heads + h) * a.max_keys + i] : i;
    const bool moves = src != i;
    EvictSlot at = {0, 0}, at_src = {0, 0};
    if (i < keep && (moves || AGED || a.weights_out)) {
        at = evict_slot(a, s, i);
        at_src = moves ? evict_slot(a, s, src) : at;
    }
    if (i < keep && a.weights_out) a.weights_out[evict_weight(a, at, h)] = a.weights[evict_weight(a, at_src, h)];
    if constexpr (AGED) {
        if (i < keep) {
            const size_t was = evict_weight(a, at_src, h);
            const long long number = evict_number(a, was, src, a.bases[head]);
            if (moves) evict_vacate(a, was);
            a.positions[evict_weight(a, at, h)] = (int)min(number, (long long)INT32_MAX);
        }
    }
    const uint32_t mask = __ballot_sync(0xffffffffu, moves);
    if (moves) {
        const int k = w0 + __popc(mask & ((1u << lane) - 1));
        auto row = [&](const EvictSlot& x) { return a.kv_pages + ((x.page * a.page_size + x.in_page) * a.num_kv_heads + h) * a.row_bytes; };
        from[k] = reinterpret_cast<const uint4*>(row(at_src));
        to[k] = reinterpret_cast<uint4*>(row(at));
    }
    __syncwarp();
    const int units = a.row_bytes / 16, all = __popc(mask) * units;
    constexpr int kAhead = 8;
    for (int j0 = lane; j0 < all; j0 += 32 * kAhead) {
        uint4 v[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int j = j0 + 32 * u;
            if (j < all) v[u] = __ldcs(from[w0 + j / units] + j % units);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int j = j0 + 32 * u;
            if (j < all) to[w0 + j / units][j % units] = v[u];
        }
    }
}

template <bool AGED>
static cudaError_t launch_kernels(EvictArgs& a, cudaStream_t stream) {
    static bool configured[64] = {};  // (by device: the attribute is the device's)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(evict_select_kernel<AGED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvictHeld * 4);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    const long long most = (long long)a.pages_per_seq * a.page_size;
    a.page_shift = (a.page_size & (a.page_size - 1)) == 0 ? __builtin_ctz(a.page_size) : -1;
    a.held = most <= kEvictHeld ? (int)most : 0;
    {
        ProfScope ps("rpa_evict_select", stream);
        evict_select_kernel<AGED><<<a.max_num_seqs * a.num_kv_heads, kEvictThreads, a.held * 4, stream>>>(a);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
    ProfScope ps("rpa_evict_move", stream);
    const int blocks = (a.max_keys - 1) / kEvictMoveThreads + 1;
    return launch_pdl(evict_move_kernel<AGED>, dim3((unsigned)a.max_num_seqs * a.num_kv_heads * blocks), dim3(kEvictMoveThreads), 0, stream,
                      !prof_enabled(), a, blocks);
}

cudaError_t launch_evict(EvictArgs& a, cudaStream_t stream) {
    return a.positions ? launch_kernels<true>(a, stream) : launch_kernels<false>(a, stream);
}

}  // namespace rpa
