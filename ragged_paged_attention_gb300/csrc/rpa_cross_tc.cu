// Cross attention (every key visible) on the 5th-generation tensor cores of sm_103a, for bf16 caches: every
// sequence of the batch, from one row of queries on.
//
//   S = Q K^T, P = 2^(c S - m), O += P V, l += sum P, out = O / l, with m a row's running maximum of
//   c S, c = sm_scale log2(e).
//
// What bounds it: per 128 x 128 block of scores the tensor pipe takes 16 MMAs of 64 cycles at D = 128
// (1024) and 12 at D = 64 (768: PV with N = 64 takes as long as with 128), and the chain from S over
// the row maximum, the exponentials and P to the next product some 1650 cycles of one warp's latencies
// and issue slots (measured by clock reads; the 32 exponentials a cycle are not what it waits for).
// So two tiles of 128 rows are in flight on every SM, each with warps of its own: while one tile's
// softmax runs, the tensor pipe works for the other. "Long" below is 4 x 4096 queries over 4096 keys, 32/8
// heads of 128: 722 us (1523 TFLOP/s) called again and again on fresh inputs, 691 in a graph on the same ones;
// shares of it are of two builds timed in turn. With a row's 128 scores in one thread no maximum is exchanged
// between warps (two warps a row quarter, half a row a thread: long 10 % slower). The causal kernel keeps one
// tile in flight, its rows split over two warps: long 24 % slower. The two tiles are
//   TILES = 2 (D = 128): 256 rows of one KV head in one CTA, which share the K/V stream;
//   TILES = 1 (D = 64): two CTAs an SM with a tile each, whose softmaxes drift apart by themselves
//              (8 x 4864 queries over 1536 keys, 20 heads: 318 us; with TILES = 2 9 % slower). It is
//              compiled for 128 registers a thread, two CTAs' worth, and spills two of them.
// Fewer bits than 32: P goes to the tensor pipe as bf16 (2^-8 of an element at most), since V is bf16 and the
// two operands of an MMA have one type, while l adds the unrounded values; exponentials are ex2.approx (2^-22).
// Scores, maxima, sums and O are float32. In the root mean square the outputs are 2.3e-3 of themselves off the
// float64 softmax, where the exact ones rounded to bf16 are 1.7e-3 off.
// Per CTA: 4 softmax warps a tile (a row a thread); then warps
//   0 .. TILES - 1: an MMA issuer a tile;
//   2: streams K (and takes the items and loads Q); 3: streams V. One 3-D tensor copy per page-sized
//      box and 64-wide panel, pages looked up one block ahead. Boxes are whole: rows past the sequence
//      in K give scores that are masked away; in V the last block's are set to zero in shared memory
//      (0 times a NaN is NaN).
// Tensor memory per tile: S (128 columns), P (64) and O (D); the next block's QK runs while the softmax
// is still at work, as soon as its scores are in registers. At D = 128 that would be 640 columns of 512:
// the two tiles take turns with one S, which holds a block's scores for the QK and the load only.
// (P over S instead, with the next QK behind PV: 1.29 us a block against 0.97 in the causal kernel.)
// Batches of few rows: a tile of one row costs what a full one does, 0.93 us a block and SM at D = 64, about
// what HBM takes for the block's keys and values (64 decodes over 1450 keys, 20 heads: 90 us, 70 at the copy
// rate). Warps without rows that skip their exponentials do not change that (92.2 us both ways) and slow long,
// whose loop they change, by 4 %.
// Barriers, all waits bounded: k/v_full, k/v_empty (rings), q_full, q_empty (Q loaded; its last QK done and,
// where the tiles share S, the scores loaded), item_full/empty (two items' numbers, handed on by the K
// warp); per tile s_full (QK done), s_free (scores loaded), p_full (P written, O rescaled), pv_done (PV read
// P and updated O), o_empty (the epilogue has read O).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "profile.h"

namespace rpa {

// An item as the warps get it: a tile's (or two tiles') rows of one KV head against `blocks` key blocks
// from block0 on, with its sequence's numbers. One of `splits` pieces leaves its result in slots of
// kCrossSlotRows rows, the pieces' one behind another from `slot` on.
struct __align__(16) CrossItem {
    int seq, head, row, q_start, n_rows, kv_len, blocks, block0, splits, split, slot, pad;
};

template <int D, int TILES>
struct CrossTc {
    static constexpr int BK = 128;
    static constexpr int DP = D / 64;                      // 64-wide panels
    static constexpr int kPanel = 128 * 128;               // 128 rows x 128 bytes
    static constexpr int kTile = DP * kPanel;              // a Q tile, or K or V of one block
    static constexpr bool ONE_S = D == 128;                // the two tiles take turns with one S buffer
    static constexpr int kCtas = TILES == 1 ? 2 : 1;       // CTAs an SM
    static constexpr int kReserve = 1024;
    static constexpr int kFit = (232448 / kCtas - kReserve * kCtas - TILES * kTile) / kTile;
    static constexpr int kSlots = kFit > 8 ? 8 : kFit;
    static constexpr int NK = kSlots / 2, NV = kSlots - NK;
    static constexpr int kOffK = TILES * kTile;
    static constexpr int kOffV = kOffK + NK * kTile;
    static constexpr int kOffBar = kOffV + NV * kTile;
    static constexpr int kBars = 2 * (NK + NV) + 9 + 5 * TILES;
    static constexpr int kOffItem = (kOffBar + kBars * 8 + 15) / 16 * 16;  // [2] CrossItem, abort, TMEM base
    static constexpr int kSmem = kOffItem + 2 * (int)sizeof(CrossItem) + 16;
    static constexpr int kSoft = 4 * TILES;                // softmax warps
    static constexpr int kThreads = (kSoft + 4) * 32;
    static constexpr int kColS = 0, kColSStep = ONE_S ? 0 : 128;
    static constexpr int kColP = ONE_S ? 128 : TILES * 128, kColO = kColP + TILES * 64;
    static constexpr int kTmemCols = TILES * 256;
    // registers: the launch's share of the SM, dealt out again by warpgroup (setmaxnreg)
    static constexpr int kRegsSoft = TILES == 1 ? 184 : 208, kRegsRest = TILES == 1 ? 72 : 88;
    static constexpr int kRegsLaunch = TILES == 1 ? 128 : 168;
    static_assert(TILES * 128 * kRegsSoft + 128 * kRegsRest <= kThreads * kRegsLaunch, "register split");
    static_assert(NK >= 1 && NV >= 1 && kSmem <= 232448 / kCtas - 1024 * (kCtas - 1), "shared memory");
    static_assert(kColO + TILES * D <= kTmemCols, "tensor memory");
};

template <int R>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// 32 bytes of eight registers in one store (p 32-byte aligned): whole sectors, half the instructions.
__device__ __forceinline__ void st_global_32b(void* p, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

template <int D, int TILES>
__global__ void __launch_bounds__(CrossTc<D, TILES>::kThreads, CrossTc<D, TILES>::kCtas)
    rpa_cross_tc_kernel(const __grid_constant__ RpaArgs a, const __grid_constant__ CUtensorMap tm_kv,
                        const __grid_constant__ CUtensorMap tm_q, int box_rows) {
    using T = CrossTc<D, TILES>;
    constexpr int BK = T::BK, NK = T::NK, NV = T::NV;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + T::kOffBar);
    uint64_t* k_empty = k_full + NK;
    uint64_t* v_full = k_empty + NK;
    uint64_t* v_empty = v_full + NV;
    uint64_t* q_full = v_empty + NV;
    uint64_t* q_empty = q_full + 1;
    uint64_t* item_full = q_full + 2;   // [2]
    uint64_t* item_empty = q_full + 4;  // [2]
    uint64_t* v_land = q_full + 6;      // the last block's V, before its rows past the sequence are zeroed
    uint64_t* fin = q_full + 7;         // every product has completed
    uint64_t* join = q_full + 8;        // tile 0's softmax warps, around a piece's ticket
    uint64_t* s_full = q_full + 9;      // [TILES] each
    uint64_t* s_free = s_full + TILES;
    uint64_t* o_empty = s_full + 2 * TILES;
    uint64_t* p_full = s_full + 3 * TILES;
    uint64_t* pv_done = s_full + 4 * TILES;
    CrossItem* s_items = reinterpret_cast<CrossItem*>(smem + T::kOffItem);
    volatile int& s_abort = *reinterpret_cast<volatile int*>(smem + T::kOffItem + 2 * sizeof(CrossItem));
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + T::kOffItem + 2 * sizeof(CrossItem) + 4);
    volatile int& s_last = *reinterpret_cast<volatile int*>(smem + T::kOffItem + 2 * sizeof(CrossItem) + 8);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    WsHeader* hdr = a.hdr;
    uint32_t* err = &hdr->error_bits;
    const int G = a.num_q_heads / a.num_kv_heads;
    constexpr int kMma0 = T::kSoft, kKw = T::kSoft + 2, kVw = T::kSoft + 3;

    if (tid == 0) {
        for (int i = 0; i < NK; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], TILES);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], TILES);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, TILES);
        mbar_init(v_land, 1);
        mbar_init(fin, TILES);
        mbar_init(join, 4);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], T::kThreads / 32);
        }
        for (int t = 0; t < TILES; ++t) {
            mbar_init(&s_full[t], 1);
            mbar_init(&s_free[t], 4);  // (softmax warps arrive once each)
            mbar_init(&p_full[t], 4);
            mbar_init(&o_empty[t], 4);
            mbar_init(&pv_done[t], 1);
        }
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMma0) tmem_alloc(tmem_slot, T::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // started early behind the plan, whose lists are complete from here on. (Nothing may start early
    // behind this grid: the next call's plan would overwrite the lists under it.)
    pdl_wait();

    uint32_t items = 0;  // items this CTA has taken (ring slots, q phases)
    // Reads the next item (every warp, or the one thread that speaks for it); false when there is none.
    auto next_item_of = [&](CrossItem& it, auto alone) -> bool {
        constexpr bool kAlone = decltype(alone)::value;
        const uint32_t slot = items & 1, ph = (items >> 1) & 1;
        it.seq = -1;
        if (mbar_wait(&item_full[slot], ph, err)) it = s_items[slot];
        if (!kAlone) __syncwarp();
        if (kAlone || lane == 0) mbar_arrive(&item_empty[slot]);
        if (it.seq < 0 || s_abort) return false;
        ++items;
        return true;
    };
    auto next_item = [&](CrossItem& it) { return next_item_of(it, std::false_type()); };

    CrossItem it;
    if (warp < T::kSoft) {
        // ---------------- softmax and epilogue: thread = row of its tile ----------------
        regs_inc<T::kRegsSoft>();
        const int t = warp >> 2, quarter = warp & 3;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t col_s = tmem + lane_off + T::kColS + t * T::kColSStep, col_p = tmem + lane_off + T::kColP + t * 64,
                       col_o = tmem + lane_off + T::kColO + t * D;
        const float cs = a.sm_scale * kLog2e;
        uint32_t nblk = 0;  // blocks this tile has processed
        uint32_t njoin = 0;
        auto join_warps = [&]() -> bool {  // a bounded barrier of the tile's four warps
            __syncwarp();
            if (lane == 0) mbar_arrive(join);
            return mbar_wait(join, njoin++ & 1, err);
        };
        bool ok = true;
        while (ok && next_item(it)) {
            if (it.row + t * 128 >= it.n_rows) continue;  // this item has no such tile
            const int R = it.row + t * 128 + quarter * 32 + lane;
            float m_use = -INFINITY, l = 0.f;
            for (int j = 0; ok && j < it.blocks; ++j, ++nblk) {
                const uint32_t par = nblk & 1;
                if (!mbar_wait(&s_full[t], par, err)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                float x[BK];
#pragma unroll
                for (int c = 0; c < BK / 32; ++c) tmem_ld32_nowait(col_s + c * 32, x + c * 32);
                tmem_ld_wait();
                tmem_landed<BK>(x);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_free[t]);
                const int valid = it.kv_len - (it.block0 + j) * BK;
                if (valid < BK) {
#pragma unroll
                    for (int i = 0; i < BK; ++i) x[i] = i < valid ? x[i] : -INFINITY;
                }
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < BK; i += 2) mx4[(i >> 1) & 3] = fmax3(mx4[(i >> 1) & 3], x[i], x[i + 1]);
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * cs;  // log2 units (cs > 0)
                // lazy: the reference maximum moves only when it has grown by more than 2^8
                const bool had = m_use > -INFINITY, rescale = mx > m_use + 8.f;
                float alpha = 1.f;
                if (rescale) {
                    alpha = fast_exp2(m_use - mx);
                    m_use = mx;
                }
                const float nmu = m_use == -INFINITY ? 0.f : -m_use;
                const bool row_rescale = rescale && had;
                if (__any_sync(0xffffffffu, row_rescale)) {
                    if (!mbar_wait(&pv_done[t], par ^ 1, err)) {  // the previous block's PV has written O
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const float f = row_rescale ? alpha : 1.f;
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t o[16];
                        tmem_ld16(col_o + c * 16, o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st16_nowait(col_o + c * 16, o);
                    }
                }
                float2 sum2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                const float2 cs2 = make_float2(cs, cs), nmu2 = make_float2(nmu, nmu);
                // the previous block's PV has read P
                ok = ok && (nblk == 0 || mbar_wait(&pv_done[t], par ^ 1, err));
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < BK / 32; ++c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float2 p = ffma2(make_float2(x[c * 32 + 2 * e], x[c * 32 + 2 * e + 1]), cs2, nmu2);
                        p.x = fast_exp2(p.x);
                        p.y = fast_exp2(p.y);
                        sum2[e & 1] = fadd2(sum2[e & 1], p);
                        pk[e] = pack_bf16(p.x, p.y);
                    }
                    tmem_st16_nowait(col_p + c * 16, pk);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[t]);
                l = l * alpha + ((sum2[0].x + sum2[1].x) + (sum2[0].y + sum2[1].y));
            }
            // epilogue: O of the last PV
            if (ok && mbar_wait(&pv_done[t], (nblk - 1) & 1, err)) {
                tc_fence_after();
                const bool rv = R < it.n_rows;
                if (it.splits > 1) {
                    // a piece: its rows' maximum (log2 units), sum and O as they are; the last piece of the
                    // head to arrive joins them all
                    const int rows16 = cdiv(it.n_rows, kCrossSlotRows) * kCrossSlotRows;
                    const size_t row = (size_t)it.slot * kCrossSlotRows + (size_t)it.split * rows16 + R;
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        float o[32];
                        tmem_ld32(col_o + c * 32, o);
                        if (rv) {
                            float4* d4 = reinterpret_cast<float4*>(a.partial_o + row * D + c * 32);
#pragma unroll
                            for (int i = 0; i < 8; ++i) d4[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                        }
                    }
                    if (rv) *reinterpret_cast<float2*>(a.partial_ml + row * 2) = make_float2(m_use, l);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&o_empty[t]);
                    __threadfence();
                    ok = join_warps();
                    if (ok && tid == 0) s_last = atomicAdd(&a.tickets[it.slot / 2], 1) == it.splits - 1;
                    ok = ok && join_warps();
                    const bool last = ok && s_last;
                    ok = ok && join_warps();  // (s_last is read before the next piece's is written)
                    if (last) {
                        __threadfence();
                        const float* ml = a.partial_ml + (size_t)it.slot * kCrossSlotRows * 2;
                        const float* po = a.partial_o + (size_t)it.slot * kCrossSlotRows * D;
                        // in one pass with a running maximum, as many of the results' loads in flight as pays:
                        // with few rows a place of 4 columns a thread and eight pieces at a time (1 query over
                        // 20000 keys: 25.2 us, four places and two pieces 28.0), else four places and two
                        // pieces (64 queries over 16384 keys, 16 heads of 64: 32 us; a place at a time, in a
                        // pass for the maxima and one for the sums, 48)
                        const int places = it.n_rows * (D / 4);
                        auto joined = [&](auto at_once, auto pieces_at_once) {
                            constexpr int U = decltype(at_once)::value, P = decltype(pieces_at_once)::value;
                            for (int i0 = tid; i0 < places; i0 += 128 * U) {
                                float M[U], L[U];
                                float4 acc[U];
#pragma unroll
                                for (int u = 0; u < U; ++u) {
                                    M[u] = -INFINITY;
                                    L[u] = 0.f;
                                    acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                                }
#pragma unroll P
                                for (int sp = 0; sp < it.splits; ++sp) {
                                    float2 m[U];
                                    float4 o[U];
#pragma unroll
                                    for (int u = 0; u < U; ++u) {
                                        const int i = min(i0 + 128 * u, places - 1), r = sp * rows16 + i / (D / 4);
                                        m[u] = __ldcg(reinterpret_cast<const float2*>(ml) + r);
                                        o[u] = __ldcg(reinterpret_cast<const float4*>(po + (size_t)r * D + i % (D / 4) * 4));
                                    }
#pragma unroll
                                    for (int u = 0; u < U; ++u) {
                                        const float Mn = fmaxf(M[u], m[u].x), Mu = Mn == -INFINITY ? 0.f : Mn;
                                        const float was = fast_exp2(M[u] - Mu), f = fast_exp2(m[u].x - Mu);
                                        M[u] = Mn;
                                        L[u] = L[u] * was + f * m[u].y;
                                        acc[u].x = acc[u].x * was + f * o[u].x;
                                        acc[u].y = acc[u].y * was + f * o[u].y;
                                        acc[u].z = acc[u].z * was + f * o[u].z;
                                        acc[u].w = acc[u].w * was + f * o[u].w;
                                    }
                                }
#pragma unroll
                                for (int u = 0; u < U; ++u) {
                                    const int i = i0 + 128 * u, r = i / (D / 4);
                                    if (i >= places) break;
                                    const float inv = L[u] > 0.f ? 1.f / L[u] : 0.f;
                                    __nv_bfloat16* dst = a.out + ((size_t)(it.q_start + r / G) * a.num_q_heads + it.head * G + r % G) * D +
                                                         i % (D / 4) * 4;
                                    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(acc[u].x * inv, acc[u].y * inv),
                                                                                pack_bf16(acc[u].z * inv, acc[u].w * inv));
                                }
                            }
                        };
                        if (places <= 128)
                            joined(std::integral_constant<int, 1>(), std::integral_constant<int, 8>());
                        else
                            joined(std::integral_constant<int, 4>(), std::integral_constant<int, 2>());
                    }
                    if (!ok) s_abort = 1;
                    continue;
                }
                // rows of 32-byte units where `out` allows them (64 sequences of 64 queries and keys, 32/8 heads of
                // 128: 30 us, in 16-byte stores 33; long 2 % slower in those)
                const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
                const float inv = l > 0.f ? 1.f / l : 0.f;
                __nv_bfloat16* dst = a.out + ((size_t)(it.q_start + (rv ? R / G : 0)) * a.num_q_heads + it.head * G +
                                              (rv ? R % G : 0)) * D;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    tmem_ld32(col_o + c * 32, o);
                    if (rv) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) pk[i] = pack_bf16(o[2 * i] * inv, o[2 * i + 1] * inv);
                        if (wide) {
                            st_global_32b(dst + c * 32, pk);
                            st_global_32b(dst + c * 32 + 16, pk + 8);
                        } else {
                            uint4* d4 = reinterpret_cast<uint4*>(dst + c * 32);
#pragma unroll
                            for (int i = 0; i < 4; ++i) d4[i] = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&o_empty[t]);
            } else {
                ok = false;
            }
            if (!ok) s_abort = 1;
        }
    } else {
        regs_dec<T::kRegsRest>();
        if (warp >= kMma0 && warp < kMma0 + TILES) {
            // ---------------- MMA issuer of tile t (a constant in either branch) ----------------
            // One lane, elected once, does all of it: the ring positions and phases are its registers, and a
            // commit tracks the products of its own thread alone. Under a test for lane 0 the compiler does
            // not know that one lane issues, and an MMA took some 80 cycles to issue (long 28 % slower).
            auto issue = [&](auto tile) {
                constexpr int t = decltype(tile)::value;
                constexpr uint32_t idesc_qk = umma_idesc_bf16(128, BK, false, false);
                constexpr uint32_t idesc_pv = umma_idesc_bf16(128, D, false, true);
                const uint64_t qdesc = umma_desc_sw128(smem_u32(smem + t * T::kTile), 16, 1024);
                const uint64_t kdesc = umma_desc_sw128(smem_u32(smem + T::kOffK), 16, 1024);
                const uint64_t vdesc = umma_desc_sw128(smem_u32(smem + T::kOffV), T::kPanel, 1024);
                const uint32_t col_s = tmem + T::kColS + t * T::kColSStep, col_p = tmem + T::kColP + t * 64, col_o = tmem + T::kColO + t * D;
                uint32_t jk = 0, jv = 0;         // ring positions
                uint32_t n_own = 0, n_other = 0;  // QKs of this tile, and of the other one before the next of these
                uint32_t npv = 0, no = 0;        // PVs, and items this tile has had
                bool ok = true;
                while (ok && next_item_of(it, std::true_type())) {
                    const bool active = it.row + t * 128 < it.n_rows, both = TILES == 2 && it.row + 128 < it.n_rows;
                    ok = mbar_wait(q_full, (items - 1) & 1, err);
                    for (int j = 0; ok && j <= it.blocks; ++j) {
                        if (j < it.blocks) {  // QK of block j
                            const uint32_t slot = jk % NK;
                            ok = mbar_wait(&k_full[slot], (jk / NK) & 1, err);
                            ++jk;
                            if (t == 1) ++n_other;  // in turn: tile 0's QK of a block, then tile 1's
                            if (active) {
                                // the scores that lie there have been read
                                if (T::ONE_S && n_other > 0) ok = ok && mbar_wait(&s_free[1 - t], (n_other - 1) & 1, err);
                                if (n_own > 0) ok = ok && mbar_wait(&s_free[t], (n_own - 1) & 1, err);
                                if (!ok) break;
                                tc_fence_after();
                                const uint64_t kb = kdesc + (uint64_t)((slot * T::kTile) >> 4);
#pragma unroll
                                for (int ks = 0; ks < D / 16; ++ks) {
                                    const uint32_t off = ((ks >> 2) * T::kPanel + (ks & 3) * 32) >> 4;
                                    umma_bf16(col_s, qdesc + off, kb + off, idesc_qk, ks > 0 ? 1u : 0u);
                                }
                                umma_commit(&s_full[t]);
                                umma_commit(&k_empty[slot]);
                                if (!T::ONE_S && j + 1 == it.blocks) umma_commit(q_empty);
                                ++n_own;
                            } else {
                                if (!ok) break;
                                mbar_arrive(&k_empty[slot]);
                                if (j + 1 == it.blocks) mbar_arrive(q_empty);
                            }
                            if (t == 0 && both) ++n_other;
                        }
                        if (T::ONE_S && active && j == it.blocks) {
                            // With S shared, Q is free once the last scores have been loaded too: the issuer
                            // that has no tile of this item follows none of the loads, and its wait for the
                            // next item's would pass at an older phase.
                            ok = mbar_wait(&s_free[t], (n_own - 1) & 1, err);
                            if (!ok) break;
                            mbar_arrive(q_empty);
                        }
                        if (j > 0) {  // PV of block j - 1
                            const uint32_t slot = jv % NV;
                            ok = mbar_wait(&v_full[slot], (jv / NV) & 1, err);
                            ++jv;
                            if (active) {
                                if (j == 1 && no > 0) ok = ok && mbar_wait(&o_empty[t], (no - 1) & 1, err);
                                const uint64_t vb = vdesc + (uint64_t)((slot * T::kTile) >> 4);
                                ok = ok && mbar_wait(&p_full[t], npv & 1, err);
                                if (!ok) break;
                                tc_fence_after();
#pragma unroll
                                for (int kk = 0; kk < BK / 16; ++kk)
                                    umma_bf16_ta(col_o, col_p + kk * 8, vb + ((kk * 16 * 128) >> 4), idesc_pv,
                                                 (j > 1 || kk > 0) ? 1u : 0u);
                                umma_commit(&pv_done[t]);
                                umma_commit(&v_empty[slot]);
                                ++npv;
                            } else {
                                if (!ok) break;
                                mbar_arrive(&v_empty[slot]);
                            }
                        }
                    }
                    if (active) ++no;
                    if (!ok) s_abort = 1;
                }
                // the products (and the arrivals committed behind them) end before shared memory goes
                umma_commit(fin);
                mbar_wait(fin, 0, err);
            };
            if (elect_one()) {
                if (warp == kMma0)
                    issue(std::integral_constant<int, 0>());
                else
                    issue(std::integral_constant<int, TILES - 1>());
            }
            __syncwarp();
        } else if (warp == kKw || warp == kVw) {
            // ---------------- K (and items, Q) and V streams ----------------
            const int part = warp == kVw;
            uint64_t* full = part ? v_full : k_full;
            uint64_t* empty = part ? v_empty : k_empty;
            const uint32_t N = part ? NV : NK;
            const int lbr = __ffs(box_rows) - 1, lps = __ffs(a.page_size) - 1, in_page = a.page_size - 1;
            const uint32_t box_bytes = (uint32_t)box_rows * 128 * T::DP;
            uint32_t jr = 0;     // ring position
            uint32_t nland = 0;  // V blocks zeroed behind their rows
            uint32_t fetched = 0;
            bool ok = true;
            const int n_items = hdr->num_items[1];
            // The first lane of the K warp hands the next item to every warp. (It takes the item once the
            // last one's copies are issued, not earlier: a CTA that held an item in reserve would keep it
            // from an idle one.)
            auto fetch = [&]() {
                const int place = atomicAdd(&hdr->next_item[1], 1);
                const uint32_t slot = fetched & 1, ph = (fetched >> 1) & 1;
                CrossItem n;
                n.seq = -1;
                if (place < n_items) {
                    const WorkItem w = a.pre_items[place];
                    n.seq = w.seq;
                    n.head = w.head;
                    n.q_start = w.key_begin;
                    n.n_rows = w.first_item;
                    n.kv_len = w.key_end;
                    n.splits = w.num_splits;
                    n.split = w.split;
                    n.row = w.num_splits > 1 ? 0 : w.row_begin;
                    n.slot = w.row_begin;
                    const int blocks = cdiv(n.kv_len, BK);  // (pieces are at least a block: the plan's bound)
                    n.block0 = (int)((long long)blocks * w.split / w.num_splits);
                    n.blocks = (int)((long long)blocks * (w.split + 1) / w.num_splits) - n.block0;
                }
                if (!mbar_wait(&item_empty[slot], ph ^ 1, err)) s_abort = 1;
                if (s_abort) n.seq = -1;
                s_items[slot] = n;
                mbar_arrive(&item_full[slot]);
                ++fetched;
            };
            while (ok) {
                if (!part && lane == 0) fetch();
                __syncwarp();
                if (!next_item(it)) break;
                const int* tbl = a.page_indices + (size_t)it.seq * a.pages_per_seq;
                auto page_of = [&](int j) -> int {
                    const int key = (it.block0 + j) * BK + lane * box_rows;
                    return (lane * box_rows < BK && j < it.blocks && key < it.kv_len) ? __ldg(tbl + (key >> lps)) : 0;
                };
                int page_next = page_of(0);
                for (int j = 0; ok && j < it.blocks; ++j, ++jr) {
                    int page = page_next;
                    page_next = page_of(j + 1);
                    const int key0 = (it.block0 + j) * BK, valid = it.kv_len - key0;  // valid >= 1
                    const int boxes = valid >= BK ? BK >> lbr : (valid + box_rows - 1) >> lbr;
                    if (lane < boxes && (unsigned)page >= (unsigned)a.total_num_pages) {
                        if (!part) set_error(err, RPA_DEV_ERR_PAGE);
                        page = 0;  // an in-bounds page keeps the barrier's byte count; the error is recorded
                    }
                    const uint32_t slot = jr % N, ph = (jr / N) & 1;
                    const bool ragged = part && valid < BK;
                    uint64_t* bar = ragged ? v_land : &full[slot];
                    int g = 1;
                    if (lane == 0) {
                        g = mbar_wait(&empty[slot], ph ^ 1, err);
                        if (g) mbar_arrive_expect_tx(bar, (uint32_t)boxes * box_bytes);
                    }
                    ok = __shfl_sync(0xffffffffu, g, 0) != 0;
                    if (!ok) break;
                    uint8_t* stage = smem + (part ? T::kOffV : T::kOffK) + slot * T::kTile;
                    if (lane < boxes) {
                        const int z = (page << lps) + ((key0 + lane * box_rows) & in_page);
#pragma unroll
                        for (int p = 0; p < T::DP; ++p)
                            tma_load_3d(smem_u32(stage + p * T::kPanel + lane * box_rows * 128), &tm_kv, 64 * p, 2 * it.head + part, z, bar);
                    }
                    if (ragged) {
                        // the rows past the sequence: zeros, whatever the page or an earlier block left there
                        ok = mbar_wait(v_land, nland & 1, err);
                        ++nland;
                        if (!ok) break;  // (every lane has waited)
                        for (int i = valid * 8 + lane; i < BK * 8; i += 32)
#pragma unroll
                            for (int p = 0; p < T::DP; ++p)
                                *reinterpret_cast<uint4*>(stage + p * T::kPanel + i * 16) = make_uint4(0, 0, 0, 0);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&full[slot]);
                    }
                    if (!part && j == 0) {
                        // the item's Q behind its first keys: it waits for the previous item's last QK
                        if (lane == 0) {
                            ok = mbar_wait(q_empty, (items & 1), err);
                            if (ok) {
                                const int tiles = min(TILES, cdiv(it.n_rows - it.row, 128));
                                mbar_arrive_expect_tx(q_full, tiles * T::kTile);
                                for (int t = 0; t < tiles; ++t)
#pragma unroll
                                    for (int p = 0; p < T::DP; ++p)
                                        tma_load_3d(smem_u32(smem + t * T::kTile + p * T::kPanel), &tm_q, 64 * p, it.head * G,
                                                    it.q_start + (it.row + t * 128) / G, q_full);
                            }
                        }
                        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                    }
                }
                if (!ok) s_abort = 1;
            }
            if (lane == 0 && s_abort) {
                // an aborted K warp still ends the other warps' wait for an item; the copies under way
                // land (bounded) before shared memory goes
                if (!part && !ok) fetch();
                for (uint32_t i = jr > N ? jr - N : 0; i < jr; ++i) mbar_wait(&full[i % N], (i / N) & 1, err);
                if (!part && items > 0) mbar_wait(q_full, (items - 1) & 1, err);
            }
            __syncwarp();
        } else {
            while (next_item(it)) {
            }
        }
    }
    // every role has left its loop
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMma0) tmem_dealloc(tmem, T::kTmemCols);
}

template <int D, int TILES>
static cudaError_t launch_cross(const RpaArgs& a, int num_sms, cudaStream_t stream, const CUtensorMap& tkv,
                                const CUtensorMap& tq, int box_rows) {
    using T = CrossTc<D, TILES>;
    auto kern = rpa_cross_tc_kernel<D, TILES>;
    static bool configured[64] = {};  // (by device: the attribute is the device's)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
        if (e != cudaSuccess) return e;
        // the warpgroups' register shares are dealt out of what the launch holds
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, kern);
        if (e != cudaSuccess) return e;
        if (fa.numRegs != T::kRegsLaunch) return cudaErrorLaunchOutOfResources;
        configured[dev] = true;
    }
    ProfScope ps("rpa_cross_tc", stream);
    return launch_pdl(kern, dim3(num_sms * T::kCtas), dim3(T::kThreads), T::kSmem, stream, a.overlap != 0, a, tkv, tq, box_rows);
}

cudaError_t launch_rpa_cross_tc(const RpaArgs& a, int num_sms, cudaStream_t stream) {
    CUtensorMap tkv, tq;
    const int ps = a.page_size, G = a.num_q_heads / a.num_kv_heads, box_rows = ps < 128 ? ps : 128;
    if (!make_tmap_bf16(&tkv, a.kv_pages, a.head_dim, 2 * a.num_kv_heads, (uint64_t)a.total_num_pages * ps, 1, box_rows) ||
        !make_tmap_bf16(&tq, a.q, a.head_dim, a.num_q_heads, a.max_num_tokens, G, 128 / G))
        return cudaErrorInvalidValue;
    return a.head_dim == 64 ? launch_cross<64, 1>(a, num_sms, stream, tkv, tq, box_rows)
                            : launch_cross<128, 2>(a, num_sms, stream, tkv, tq, box_rows);
}

int rpa_cross_tile_rows(const RpaArgs& a) { return a.head_dim == 64 ? 128 : 256; }

bool rpa_cross_tc_takes(const RpaArgs& a) {
    const int G = a.num_q_heads / a.num_kv_heads, ps = a.page_size;
    return !a.causal && !a.kv_byte && !a.has_scale && a.soft_cap == 0.f && a.sm_scale > 0.f &&
           (a.head_dim == 64 || a.head_dim == 128) && (ps & (ps - 1)) == 0 && ps >= 8 && 128 % G == 0;
}

}  // namespace rpa
