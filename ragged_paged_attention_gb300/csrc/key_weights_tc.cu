// Key weights of sequences with more than 16 query rows a KV head (windows of a prompt's last queries, whole prompts) over
// bf16 caches, on the 5th-generation tensor cores of sm_103a.
//
// Two kernels of one frame: a tile of 128 query rows (token, q head) stays, K's blocks of 128 keys go by, and two groups of
// four warps take the even and the odd blocks' scores, each from a buffer of tensor memory of its own.
//   STATS: S = Q K^T, a row a thread: its running maximum and sum over a piece of its keys, one result a group.
//   SUM:   S^T = K Q^T, a key a thread: the sum over the tile's rows of 2^(c s - L), L = log2 of the row's sum, joined from its
//          pieces' results; over all tiles of the sequence, in registers, for a chunk of up to 8 blocks.
// A block of 128 x 128 scores is 512 cycles of the tensor pipe and of the exponentials (D = 128) and 32 KB of K, which
// HBM brings in some 700: both kernels are bound by reading K where a sequence has one tile, by the exponentials where
// it has many. 8 windows of 32 queries over 8000-16000 keys, 32/8 heads of 128: STATS 45 us, SUM 53 (185 MB of K each: 4.1
// and 3.5 TB/s with one tile in flight an SM); 16 rows at a time on mma.sync 252 and 326 us. With a soft cap
// (tanhf) 102 and 137 us, 401 and 464 there. A block's 128 scores a thread fill the registers: of 168, SUM spills 16 bytes, with
// the cap's 128 unrolled tanhf 168 (STATS 56). Scores are exact products summed in float32; maxima, sums and L are float32.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "profile.h"

namespace rpa {

template <int D>
struct KwTc {
    static constexpr int DP = D / 64;
    static constexpr int kPanel = 128 * 128, kTile = DP * kPanel;   // 128 rows of Q, or 128 keys
    static constexpr int NQ = D == 256 ? 1 : 2, NK = D == 256 ? 2 : 4;
    static constexpr int kOffK = NQ * kTile;
    static constexpr int kOffL = kOffK + NK * kTile;                // [8 warps][128] floats
    static constexpr int kOffBar = kOffL + 8 * 128 * 4;
    static constexpr int kBars = 2 * (NQ + NK) + 8 + 1;
    static constexpr int kOffItem = (kOffBar + kBars * 8 + 15) / 16 * 16;
    static constexpr int kSmem = kOffItem + 2 * 48 + 16;
    static constexpr int kThreads = 12 * 32;                        // 8 score warps, MMA issuer, copies, two idle
    static_assert(kSmem <= 232448, "shared memory");
};

// An item as the warps get it: row tiles [tile0, tile1) against key blocks [block0, block1) of one KV head. index: STATS'
// place of its results; first: SUM's place of the head's first result.
struct __align__(16) KwTcItem {
    int seq, head, q_start, q_len, kv_len, tile0, tile1, block0, block1, index, pieces, pad;
};

// Key blocks [lo, hi) that rows row0 .. row0 + 127 see, within [b0, b1).
__device__ __forceinline__ void kw_tc_blocks(const KwArgs& a, const KwTcItem& it, int G, int tile, int& lo, int& hi) {
    const int row0 = tile * 128, last = min(it.q_len * G, row0 + 128) - 1, p0 = it.kv_len - it.q_len + row0 / G;
    const int end = it.kv_len - it.q_len + last / G + 1, first = a.sliding_window > 0 ? max(0, p0 - a.sliding_window + 1) : 0;
    lo = max(it.block0, first >> 7);
    hi = max(lo, min(it.block1, (end + 127) >> 7));
}

template <int D, bool SUM, bool CAP>
__global__ void __launch_bounds__(KwTc<D>::kThreads, 1)
    kw_tc_kernel(const __grid_constant__ KwArgs a, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv, int q_tma,
                 int box_rows) {
    using T = KwTc<D>;
    constexpr int NQ = T::NQ, NK = T::NK;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + T::kOffBar);
    uint64_t* k_empty = k_full + NK;
    uint64_t* q_full = k_empty + NK;
    uint64_t* q_empty = q_full + NQ;
    uint64_t* s_full = q_empty + NQ;         // [2] a buffer of scores each
    uint64_t* s_free = s_full + 2;
    uint64_t* item_full = s_full + 4;
    uint64_t* item_empty = s_full + 6;
    uint64_t* fin = s_full + 8;
    KwTcItem* s_items = reinterpret_cast<KwTcItem*>(smem + T::kOffItem);
    volatile int& s_abort = *reinterpret_cast<volatile int*>(smem + T::kOffItem + 2 * sizeof(KwTcItem));
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + T::kOffItem + 2 * sizeof(KwTcItem) + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = a.num_q_heads / a.num_kv_heads;
    uint32_t* err = &a.hdr->error_bits;
    constexpr int kMma = 8, kCopy = 9;
    if (tid == 0) {
        for (int i = 0; i < NK; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < NQ; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_free[i], 4);
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], 10);  // (the idle warps take no items)
        }
        mbar_init(fin, 1);
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMma) tmem_alloc(tmem_slot, 256);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (!SUM) pdl_launch_dependents();  // (the kernels behind wait for this grid's end)
    pdl_wait();
    uint32_t items = 0;
    auto next_item = [&](KwTcItem& it, bool alone) -> bool {
        const uint32_t slot = items & 1, ph = (items >> 1) & 1;
        it.seq = -1;
        if (mbar_wait(&item_full[slot], ph, err)) it = s_items[slot];
        if (!alone) __syncwarp();
        if (alone || lane == 0) mbar_arrive(&item_empty[slot]);
        if (it.seq < 0 || s_abort) return false;
        ++items;
        return true;
    };
    KwTcItem it;
    if (warp < 8) {
        // ---------------- scores: this group's buffer ----------------
        const int group = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t col_s = tmem + ((uint32_t)(quarter * 32) << 16) + group * 128;
        const float cs = CAP ? kLog2e : a.sm_scale * kLog2e;  // (> 0: the host's condition)
        [[maybe_unused]] const float cap = a.soft_cap, to_cap = a.sm_scale / a.soft_cap;
        float* Ls = reinterpret_cast<float*>(smem + T::kOffL) + warp * 128;  // (a warp's own copy: no warp waits for another)
        uint32_t mine = 0;  // blocks of this group so far
        bool ok = true;
        // this group's next scores in registers; false on a timeout
        float x[128];
        auto load = [&]() -> bool {
            if (!mbar_wait(&s_full[group], mine & 1, err)) return false;
            ++mine;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32_nowait(col_s + c * 32, x + c * 32);
            tmem_ld_wait();
            tmem_landed<128>(x);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_free[group]);
            if constexpr (CAP) {
#pragma unroll
                for (int i = 0; i < 128; ++i) x[i] = cap * tanhf(x[i] * to_cap);
            }
            return true;
        };
        while (ok && next_item(it, false)) {
            if constexpr (!SUM) {
                const int R = it.tile0 * 128 + r;
                const bool rv = R < it.q_len * G;
                const int qpos = rv ? it.kv_len - it.q_len + R / G : -1, wlo = a.sliding_window > 0 ? qpos - a.sliding_window + 1 : 0;
                float m = -INFINITY, l = 0.f;
                int lo, hi;
                kw_tc_blocks(a, it, G, it.tile0, lo, hi);
                for (int b = lo + ((lo ^ group) & 1); ok && b < hi; b += 2) {
                    ok = load();
                    if (!ok) break;
                    const int c0 = wlo - b * 128, c1 = qpos - b * 128;  // columns [c0, c1] are seen
                    if (__any_sync(0xffffffffu, c0 > 0 || c1 < 127)) {
#pragma unroll
                        for (int i = 0; i < 128; ++i) x[i] = i >= c0 && i <= c1 ? x[i] : -INFINITY;
                    }
                    float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < 128; i += 2) mx4[(i >> 1) & 3] = fmax3(mx4[(i >> 1) & 3], x[i], x[i + 1]);
                    const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * cs;
                    if (mx > m) {
                        l *= fast_exp2(m - mx);
                        m = mx;
                    }
                    const float nm = m == -INFINITY ? 0.f : -m;
                    const float2 cs2 = make_float2(cs, cs), nm2 = make_float2(nm, nm);
                    float2 sum2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int i = 0; i < 128; i += 2) {
                        float2 p = ffma2(make_float2(x[i], x[i + 1]), cs2, nm2);
                        p.x = fast_exp2(p.x);
                        p.y = fast_exp2(p.y);
                        sum2[(i >> 1) & 1] = fadd2(sum2[(i >> 1) & 1], p);
                    }
                    l += (sum2[0].x + sum2[1].x) + (sum2[0].y + sum2[1].y);
                }
                if (ok) a.tc_stats[((size_t)it.index * 2 + group) * 128 + r] = make_float2(m, l);
            } else {
                // this thread's key of each block of this group's, over the rows of all tiles
                constexpr int kW = kKwTcChunk / 2 + 1;
                const int w0 = it.block0 >> 1;
                float w[kW] = {};
                for (int tile = it.tile0; ok && tile < it.tile1; ++tile) {
                    int lo, hi;
                    kw_tc_blocks(a, it, G, tile, lo, hi);
                    lo += (lo ^ group) & 1;
                    if (lo >= hi) continue;
                    // -L of the tile's rows, four a lane
                    const int tiles = cdiv(it.q_len * G, 128), rows = min(128, it.q_len * G - tile * 128);
                    const float2* st = a.tc_stats + ((size_t)it.index + ((size_t)it.head * tiles + tile) * it.pieces) * 256 + lane;
                    __syncwarp();  // (the last tile's are read)
                    float M[4], sum[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        M[k] = -INFINITY;
                        sum[k] = 0.f;
                    }
#pragma unroll 8
                    for (int i = 0; i < 2 * it.pieces; ++i) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 v = st[(size_t)i * 128 + 32 * k];
                            const float n = fmaxf(M[k], v.x), u = n == -INFINITY ? 0.f : n;
                            sum[k] = sum[k] * fast_exp2(M[k] - u) + v.y * fast_exp2(v.x - u);
                            M[k] = n;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) Ls[lane + 32 * k] = sum[k] > 0.f ? -(M[k] + log2f(sum[k])) : 0.f;  // (0: a row that is not there, whose x is -inf)
                    __syncwarp();
                    const int p0 = it.kv_len - it.q_len;
                    for (int b = lo; ok && b < hi; b += 2) {
                        ok = load();
                        if (!ok) break;
                        // rows [c0, c1) of the tile see this thread's key: token t does where p0 + t >= key > p0 + t - window.
                        // (Rows that are not there, whatever lies in them, are left out.)
                        const long long key = b * 128 + r;
                        const int c0 = (int)max((key - p0) * G - tile * 128, -1ll);
                        const int c1 = a.sliding_window > 0 ? (int)min((key - p0 + a.sliding_window) * G - tile * 128, (long long)rows) : rows;
                        if (__any_sync(0xffffffffu, c0 > 0 || c1 < 128)) {
#pragma unroll
                            for (int i = 0; i < 128; ++i) x[i] = i >= c0 && i < c1 ? x[i] : -INFINITY;
                        }
                        const float2 cs2 = make_float2(cs, cs);
                        float2 sum2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                        for (int i = 0; i < 128; i += 4) {
                            const float4 L4 = *reinterpret_cast<const float4*>(Ls + i);
                            float2 p = ffma2(make_float2(x[i], x[i + 1]), cs2, make_float2(L4.x, L4.y));
                            float2 q = ffma2(make_float2(x[i + 2], x[i + 3]), cs2, make_float2(L4.z, L4.w));
                            p.x = fast_exp2(p.x);
                            p.y = fast_exp2(p.y);
                            q.x = fast_exp2(q.x);
                            q.y = fast_exp2(q.y);
                            sum2[0] = fadd2(sum2[0], p);
                            sum2[1] = fadd2(sum2[1], q);
                        }
                        const float add = (sum2[0].x + sum2[1].x) + (sum2[0].y + sum2[1].y);
#pragma unroll
                        for (int i = 0; i < kW; ++i) w[i] += (b >> 1) - w0 == i ? add : 0.f;
                    }
                }
                const int* tbl = a.page_indices + (size_t)it.seq * a.pages_per_seq;
#pragma unroll
                for (int i = 0; i < kW; ++i) {
                    const int b = 2 * (w0 + i) + group, key = b * 128 + r;
                    if (!ok || b < it.block0 || b >= it.block1 || key >= it.kv_len) continue;
                    const int pg = key / a.page_size, page = tbl[pg];
                    if ((unsigned)page < (unsigned)a.total_num_pages) {
                        const size_t o = ((size_t)page * a.num_kv_heads + it.head) * a.page_size + (key - pg * a.page_size);
                        a.weights_out[o] = a.keep == 0.f ? w[i] : fmaf(a.keep, a.weights[o], w[i]);
                    }
                }
            }
            if (!ok) s_abort = 1;
        }
    } else if (warp == kMma) {
        if (elect_one()) {
            constexpr uint32_t idesc = umma_idesc_bf16(128, 128, false, false);
            const uint64_t qdesc = umma_desc_sw128(smem_u32(smem), 16, 1024), kdesc = umma_desc_sw128(smem_u32(smem + T::kOffK), 16, 1024);
            uint32_t jk = 0, jq = 0, used[2] = {0, 0};
            bool ok = true;
            while (ok && next_item(it, true)) {
                for (int tile = it.tile0; ok && tile < it.tile1; ++tile) {
                    int lo, hi;
                    kw_tc_blocks(a, it, G, tile, lo, hi);
                    if (lo >= hi) continue;
                    const uint32_t qs = jq % NQ;
                    ok = mbar_wait(&q_full[qs], (jq / NQ) & 1, err);
                    ++jq;
                    for (int b = lo; ok && b < hi; ++b, ++jk) {
                        const uint32_t slot = jk % NK, buf = b & 1, n = buf ? used[1]++ : used[0]++;
                        ok = mbar_wait(&k_full[slot], (jk / NK) & 1, err) && (n == 0 || mbar_wait(&s_free[buf], (n - 1) & 1, err));
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t q0 = qdesc + (uint64_t)((qs * T::kTile) >> 4), k0 = kdesc + (uint64_t)((slot * T::kTile) >> 4);
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks) {
                            const uint32_t off = ((ks >> 2) * T::kPanel + (ks & 3) * 32) >> 4;
                            if (SUM)
                                umma_bf16(tmem + buf * 128, k0 + off, q0 + off, idesc, ks > 0 ? 1u : 0u);
                            else
                                umma_bf16(tmem + buf * 128, q0 + off, k0 + off, idesc, ks > 0 ? 1u : 0u);
                        }
                        umma_commit(&s_full[buf]);
                        umma_commit(&k_empty[slot]);
                    }
                    umma_commit(&q_empty[qs]);
                }
                if (!ok) s_abort = 1;
            }
            umma_commit(fin);
            mbar_wait(fin, 0, err);
        }
        __syncwarp();
    } else if (warp == kCopy) {
        // ---------------- items, Q and K ----------------
        const int n_items = a.tc[SUM ? 1 : 0], num = a.hdr->num_items[2], piece = a.tc[2], chunk = a.tc[3];
        int* const counter = a.tc + (SUM ? 5 : 4);
        const int lbr = __ffs(box_rows) - 1, lps = __ffs(a.page_size) - 1, in_page = a.page_size - 1;
        uint32_t jk = 0, jq = 0, fetched = 0;
        auto fetch = [&]() {  // (the whole warp)
            const uint32_t slot = fetched & 1, ph = (fetched >> 1) & 1;
            KwTcItem n;
            n.seq = -1;
            int i = n_items;
            if (lane == 0 && !s_abort) i = atomicAdd(counter, 1);
            i = __shfl_sync(0xffffffffu, i, 0);
            if (i < n_items) {
                int first;
                n.seq = kw_find(SUM ? a.ends_e : a.ends_d, num, i, first);
                n.q_start = a.cu_q_lens[n.seq];
                n.q_len = a.cu_q_lens[n.seq + 1] - n.q_start;
                n.kv_len = a.kv_lens[n.seq];
                const int tiles = cdiv(n.q_len * G, 128), blocks = cdiv(n.kv_len, 128), rel = i - first;
                n.pieces = cdiv(blocks, piece);
                if (SUM) {
                    const int chunks = cdiv(blocks, chunk);
                    n.head = rel / chunks;
                    n.tile0 = 0;
                    n.tile1 = tiles;
                    n.block0 = rel % chunks * chunk;
                    n.block1 = min(blocks, n.block0 + chunk);
                    n.index = n.seq > 0 ? a.ends_d[n.seq - 1] : 0;
                } else {
                    n.index = i;
                    n.head = rel / (tiles * n.pieces);
                    n.tile0 = rel / n.pieces % tiles;
                    n.tile1 = n.tile0 + 1;
                    n.block0 = rel % n.pieces * piece;
                    n.block1 = min(blocks, n.block0 + piece);
                }
            }
            if (lane == 0) {
                if (!mbar_wait(&item_empty[slot], ph ^ 1, err)) {
                    s_abort = 1;
                    n.seq = -1;
                }
                s_items[slot] = n;
                mbar_arrive(&item_full[slot]);
            }
            ++fetched;
            __syncwarp();
        };
        bool ok = true;
        while (ok) {
            fetch();
            if (!__all_sync(0xffffffffu, next_item(it, false))) break;
            const int* tbl = a.page_indices + (size_t)it.seq * a.pages_per_seq;
            for (int tile = it.tile0; ok && tile < it.tile1; ++tile) {
                int lo, hi;
                kw_tc_blocks(a, it, G, tile, lo, hi);
                if (lo >= hi) continue;
                const uint32_t qs = jq % NQ;
                ok = __all_sync(0xffffffffu, mbar_wait(&q_empty[qs], ((jq / NQ) & 1) ^ 1, err));
                if (!ok) break;
                if (q_tma) {
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&q_full[qs], T::kTile);
#pragma unroll
                        for (int p = 0; p < T::DP; ++p)
                            tma_load_3d(smem_u32(smem + qs * T::kTile + p * T::kPanel), &tm_q, 64 * p, it.head * G, it.q_start + tile * 128 / G,
                                        &q_full[qs]);
                    }
                } else {
                    // a group size that does not divide a tile: 16 bytes at a time, rows that are not there as zeros (8 windows with 48/8
                    // heads: 321 us; on mma.sync 855)
                    for (int i = lane; i < 128 * (D / 8); i += 32) {
                        const int tr = i / (D / 8), c = i % (D / 8), R = tile * 128 + tr;
                        const bool rv = R < it.q_len * G;
                        cp_async16(smem_u32(smem + qs * T::kTile + (c >> 3) * T::kPanel + tr * 128 + (((c & 7) ^ (tr & 7)) << 4)),
                                   a.q + ((size_t)(it.q_start + (rv ? R / G : 0)) * a.num_q_heads + it.head * G + (rv ? R % G : 0)) * D + c * 8, rv);
                    }
                    cp_async_commit();
                    cp_async_wait<0>();
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&q_full[qs]);
                }
                ++jq;
                auto page_of = [&](int b) -> int {
                    const int key = b * 128 + lane * box_rows;
                    return lane * box_rows < 128 && b < hi && key < it.kv_len ? __ldg(tbl + (key >> lps)) : 0;
                };
                int page_next = page_of(lo);
                for (int b = lo; b < hi; ++b, ++jk) {
                    int page = page_next;
                    page_next = page_of(b + 1);
                    const int key0 = b * 128, valid = min(128, it.kv_len - key0), boxes = (valid + box_rows - 1) >> lbr;
                    if (lane < boxes && (unsigned)page >= (unsigned)a.total_num_pages) {
                        set_error(err, RPA_DEV_ERR_PAGE);
                        page = 0;  // an in-bounds page keeps the barrier's byte count; the error is recorded
                    }
                    const uint32_t slot = jk % NK;
                    ok = __all_sync(0xffffffffu, mbar_wait(&k_empty[slot], ((jk / NK) & 1) ^ 1, err));
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&k_full[slot], (uint32_t)(boxes * box_rows * 128 * T::DP));
                    __syncwarp();
                    if (lane < boxes) {
                        const int z = (page << lps) + ((key0 + lane * box_rows) & in_page);
#pragma unroll
                        for (int p = 0; p < T::DP; ++p)
                            tma_load_3d(smem_u32(smem + T::kOffK + slot * T::kTile + p * T::kPanel + lane * box_rows * 128), &tm_kv, 64 * p,
                                        2 * it.head, z, &k_full[slot]);
                    }
                }
            }
            if (!ok) s_abort = 1;
        }
        if (__any_sync(0xffffffffu, s_abort)) {
            // the other warps' wait for an item ends, and copies under way land (bounded) before shared memory goes
            fetch();
            if (lane == 0) {
                for (uint32_t i = jk > NK ? jk - NK : 0; i < jk; ++i) mbar_wait(&k_full[i % NK], (i / NK) & 1, err);
                for (uint32_t i = jq > NQ ? jq - NQ : 0; i < jq; ++i) mbar_wait(&q_full[i % NQ], (i / NQ) & 1, err);
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMma) tmem_dealloc(tmem, 256);
}

template <int D, bool SUM, bool CAP>
static cudaError_t launch_tc(const KwArgs& a, int num_sms, cudaStream_t stream, const CUtensorMap& tq, const CUtensorMap& tkv, int q_tma, int box_rows) {
    using T = KwTc<D>;
    auto kern = kw_tc_kernel<D, SUM, CAP>;
    static bool configured[64] = {};  // (by device: the attribute is the device's)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    ProfScope ps(SUM ? "rpa_kw_tc_sum" : "rpa_kw_tc_stats", stream);
    return launch_pdl(kern, dim3(num_sms), dim3(T::kThreads), T::kSmem, stream, !prof_enabled(), a, tq, tkv, q_tma, box_rows);
}

bool kw_tc_takes(const KwArgs& a, int head_dim, bool g4) {
    const int ps = a.page_size;
    return !g4 && (a.soft_cap != 0.f || a.sm_scale > 0.f) && (head_dim == 64 || head_dim == 128 || head_dim == 256) &&
           (ps & (ps - 1)) == 0 && ps >= 8 && (long long)a.total_num_pages * ps <= INT32_MAX;
}

cudaError_t launch_kw_tc(const KwArgs& a, int head_dim, bool sum, int num_sms, cudaStream_t stream) {
    CUtensorMap tq, tkv;
    memset(&tq, 0, sizeof tq);
    const int G = a.num_q_heads / a.num_kv_heads, ps = a.page_size, box_rows = ps < 128 ? ps : 128, q_tma = 128 % G == 0;
    if (!make_tmap_bf16(&tkv, a.kv_pages, head_dim, 2 * a.num_kv_heads, (uint64_t)a.total_num_pages * ps, 1, box_rows) ||
        (q_tma && !make_tmap_bf16(&tq, a.q, head_dim, a.num_q_heads, a.max_num_tokens, G, 128 / G)))
        return cudaErrorInvalidValue;
    auto launch = [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        if (a.soft_cap != 0.f)
            return sum ? launch_tc<D, true, true>(a, num_sms, stream, tq, tkv, q_tma, box_rows)
                       : launch_tc<D, false, true>(a, num_sms, stream, tq, tkv, q_tma, box_rows);
        return sum ? launch_tc<D, true, false>(a, num_sms, stream, tq, tkv, q_tma, box_rows)
                   : launch_tc<D, false, false>(a, num_sms, stream, tq, tkv, q_tma, box_rows);
    };
    switch (head_dim) {
        case 64: return launch(std::integral_constant<int, 64>());
        case 128: return launch(std::integral_constant<int, 128>());
        case 256: return launch(std::integral_constant<int, 256>());
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace rpa
