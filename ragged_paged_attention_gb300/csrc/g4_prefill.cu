// Prefill-class attention over the 4-bit cache (rpa_g4_forward: sequences of more than 16 query rows a KV head) on the
// 5th-generation tensor cores of sm_103a.
//
//   S = Q K^T, P = 2^(c S - m + 7), O += P V, l += sum P, out = O / l, K = s n + m rounded to bf16
//   (2^-8 of a value at most, as a bf16 cache holds it), V = s n + m rounded to f16 (or bf16: g4_fits_f16).
//
// Tiles of 128 rows (token, q head of the group; a row a thread), blocks of 64 keys. A block's 4-bit rows of the KV head
// come to shared memory by tensor copies (a page or a part of one each); four warps turn them into the 16-bit panels that
// the products read, a thread a row of K or of V: each pair of numbers is masked out as a pair of subnormals, and one
// fused multiply-add gives both values, rounded once. Two tiles of a KV head (head_dim 64 and 128) share each
// converted block, and while one's softmax runs the tensor pipe works for the other; at head_dim 256 tensor memory
// holds one tile.
// Warps: 4 softmax warps a tile; an MMA issuer a tile; one that takes items and loads Q; one that copies raw rows; 2
// converters for K and 2 for V.
// Barriers, all waits bounded: raw_full/empty, k/v_full, k/v_empty (panels), q_full, q_empty, item_full/empty; per tile
// s_full (QK done), s_free (scores loaded), and P buffer p_full (P written, O rescaled) and pv_done; per tile o_empty.
//
// What bounds it: the prompts' products alone would take 285 us at cuBLAS's rate where 4 x 4096 tokens over their own 4096 keys (32
// heads of 128, 8 KV heads) take 519 in a graph: a block's softmax (64 exponentials a row, on one of four quarters of the SM) and the conversions
// (26 cycles of such a quarter for 8 numbers of 32 rows of K, 18 of V) each take about as long as the
// products, share the issue slots, and read or write shared memory beside the tensor pipe. Without the conversions: 478 us.
// 128-key blocks had 387 without them, but no room for raw rows by tensor copies. With a soft cap and a window of 4096, 2 x
// 1024 tokens of 256 over up to 5120 keys: 207 us.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "common.cuh"
#include "g4.cuh"
#include "kernels.h"
#include "profile.h"

namespace rpa {

struct __align__(16) G4Item {
    int seq, head, row, q_start, q_len, kv_len, block0, blocks, place;
};

template <int D>
struct G4Pre {
    static constexpr int TILES = D == 256 ? 1 : 2;
    static constexpr int BK = 64;
    static constexpr int DP = D / 64;                      // 64-wide panels
    static constexpr int kQPanel = 128 * 128, kQTile = DP * kQPanel;
    static constexpr int kPanel = BK * 128, kTile = DP * kPanel;
    static constexpr int NK = D == 256 ? 2 : 4, NV = D == 256 ? 1 : 4;  // rings of blocks of K and V
    static constexpr int PB = 2;            // P buffers a tile
    static constexpr int NR = 3;                           // raw blocks on their way
    static constexpr int kRaw = BK * G4<D>::kRow;
    static constexpr int kOffK = TILES * kQTile;
    static constexpr int kOffV = kOffK + NK * kTile;
    static constexpr int kOffRaw = kOffV + NV * kTile;
    static constexpr int kOffBar = kOffRaw + NR * kRaw;
    static constexpr int kBars = 2 * (NK + NV + NR) + 9 + (3 + 2 * PB) * TILES;
    static constexpr int kOffItem = (kOffBar + kBars * 8 + 15) / 16 * 16;  // [2] G4Item, abort, TMEM base, exit, first item to do again
    static constexpr int kOffFits = kOffItem + 2 * (int)sizeof(G4Item) + 16;  // [2][2] int
    static constexpr int kSmem = kOffFits + 16;
    static constexpr int kSoft = 4 * TILES;
    static constexpr int kThreads = (kSoft + 8) * 32;
    static constexpr int kColS = 0;
    static constexpr int kColP = TILES * BK, kColO = kColP + TILES * PB * (BK / 2);
    static constexpr int kTmemCols = 512;
    // registers: the launch's share of the SM, dealt out again by warpgroup (setmaxnreg)
    static constexpr int kRegsLaunch = TILES == 2 ? 128 : 168;
    static constexpr int kRegsSoft = 184, kRegsRest = 72;
    static_assert(TILES == 1 || 256 * kRegsSoft + 256 * kRegsRest <= kThreads * kRegsLaunch, "register split");
    static_assert(kSmem <= 232448 && kOffK % 1024 == 0 && kOffV % 1024 == 0 && kOffRaw % 128 == 0 && kRaw % 128 == 0 && kOffBar % 8 == 0, "shared memory");
    static_assert(kColO + TILES * D <= kTmemCols, "tensor memory");
};

// The keys that rows of the item see: [begin, end).
__device__ __forceinline__ int g4_key_begin(const G4Item& it, int G, int window) {
    return window > 0 ? it.kv_len - it.q_len + it.row / G - window + 1 : 0;
}
__device__ __forceinline__ int g4_key_end(const G4Item& it, int G, int tiles) {
    return it.kv_len - it.q_len + (min(it.row + 128 * tiles, it.q_len * G) - 1) / G + 1;
}

template <int R>
__device__ __forceinline__ void g4_regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void g4_regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// Panels hold values times kDown. A number with all other bits of its half masked away is the bf16 subnormal n 2^-133 (or n
// 2^-129 in bits 4-7), so that one fused multiply-add with (s 2^80, m 2^-53) gives (s n + m) 2^-53, rounded once, with
// bf16's exponents: scores and outputs take the 2^53 back. (Numbers as 128 + n, and a subtraction before the multiply-add:
// 34 cycles of a quarter of the SM for 8 of them, where K's take 26 and V's 18.)
constexpr float kDown = 0x1p-53f;
__device__ __forceinline__ uint32_t bf16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t f16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
// V's panels and the P that meets them are f16 where an item's groups of V allow it. A number alone is the f16 subnormal
// n 2^-24 (or n 2^-20), and values are held times 2^-10: within 2^-11 of themselves from 2^-4 on (bf16: 2^-8), and below that,
// as f16 subnormals, within 2^-15 (twice either where |m| < 2^-7, since m is rounded first). A group fits with s < 4 (s 2^14 is a
// factor), |m| < 2^20, and s >= 2^-9 or |m| >= 2^-6, or as zeros. At the least s a step of f16 is s / 32, beside the s that the
// cache rounds to, and outputs are as near as with bf16: 2.85e-3 of themselves with s from 2^-9 to 1.5 2^-9 about zero, 2.8e-3
// in bf16 just below, 2.2e-3 with s from 2^-8 on (1.6e-3 are the outputs' own rounding). V's converters look at the groups on
// their way; an item in which one does not fit is done again with bf16 (2^-53 of V, 2^43 of P: the same 2^-10), which
// makes such a cache's prompts twice as long (4 x 4096 tokens 1016 us, not 519; one key of small V that all see is enough). (Looked at block by block before its V is turned: 4 x 4096 prompts 552 us, not 497.)
constexpr float kDownV = 0x1p-10f;
// P and l are held times 2^7: at most 2^15 (the reference maximum may lag by 2^8), and f16 keeps 8 bits of weights down to
// 2^-24 of a row's greatest (behind a first key of nearly all the weight and hardly any value, the others count).
constexpr float kUpP = 7.f;
__device__ __forceinline__ bool g4_fits_f16(uint32_t sm) {
    const uint32_t s = sm & 0xffffu, m = (sm >> 16) & 0x7fffu;
    return s < 0x4080u && m < 0x4980u && (s >= 0x3b00u || m >= 0x3c80u || (s | m) == 0);
}
// 8 numbers in order (K, whose dims lie as Q's do): byte e's two go to the low bits of two halves.
__device__ __forceinline__ uint4 g4_panel8(uint32_t w, uint32_t s2, uint32_t m2) {
    const uint32_t h = w >> 4;
    uint32_t r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = __byte_perm(w, h, e | (e << 4) | ((4 + e) << 8) | ((4 + e) << 12)) & 0x000f000fu;
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = bf16x2_fma(r[e], s2, m2);
    return make_uint4(r[0], r[1], r[2], r[3]);
}
// In the order 0, 4, 1, 5, 2, 6, 3, 7 (V, whose dims are O's columns: the epilogue puts them in order).
__device__ __forceinline__ uint4 g4_panel8_v(uint32_t w, uint32_t s2, uint32_t s2_16, uint32_t m2) {
    const uint32_t h = w >> 8;
    return make_uint4(bf16x2_fma(w & 0x000f000fu, s2, m2), bf16x2_fma(w & 0x00f000f0u, s2_16, m2), bf16x2_fma(h & 0x000f000fu, s2, m2),
                      bf16x2_fma(h & 0x00f000f0u, s2_16, m2));
}

__device__ __forceinline__ uint4 g4_panel8_v_f16(uint32_t w, uint32_t s2, uint32_t s2_16, uint32_t m2) {
    const uint32_t h = w >> 8;
    return make_uint4(f16x2_fma(w & 0x000f000fu, s2, m2), f16x2_fma(w & 0x00f000f0u, s2_16, m2), f16x2_fma(h & 0x000f000fu, s2, m2),
                      f16x2_fma(h & 0x00f000f0u, s2_16, m2));
}

template <int D, bool CAP>
__global__ void __launch_bounds__(G4Pre<D>::kThreads, 1)
    g4_prefill_kernel(const __grid_constant__ RpaArgs a, const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_kv, int q_tma, int box_rows, int tail) {
    using T = G4Pre<D>;
    using F = G4<D>;
    constexpr int BK = T::BK, NK = T::NK, NV = T::NV, TILES = T::TILES, NR = T::NR, PB = T::PB;
    // first launch (tail == 0): started early behind the plan, it waits for it, then lets the decode grid behind
    // start; only the plan's share of its CTAs works. Either launch leaves at once when the list is empty.
    if (!tail) {
        pdl_wait();
        pdl_launch_dependents();
    }
    extern __shared__ __align__(1024) uint8_t smem[];
    volatile int* flags = reinterpret_cast<volatile int*>(smem + T::kOffItem + 2 * sizeof(G4Item));
    volatile int& s_abort = flags[0];
    volatile int* item_fits = reinterpret_cast<volatile int*>(smem + T::kOffFits);  // V of item n (n & 1) in f16, by V converter
    volatile int& s_again = flags[3];
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + T::kOffItem + 2 * sizeof(G4Item) + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    WsHeader* hdr = a.hdr;
    if (tid == 0)  // one decision for the whole CTA
        flags[2] = (!tail && (int)blockIdx.x >= hdr->prefill_ctas) || *(volatile const int*)&hdr->next_item[1] >= hdr->num_items[1];
    __syncthreads();
    if (flags[2]) return;
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + T::kOffBar);
    uint64_t* k_empty = k_full + NK;
    uint64_t* v_full = k_empty + NK;
    uint64_t* v_empty = v_full + NV;
    uint64_t* raw_full = v_empty + NV;
    uint64_t* raw_empty = raw_full + NR;
    uint64_t* turned = raw_empty + NR;  // [2]: V's converters have ended item n (n & 1)
    uint64_t* q_full = turned + 2;
    uint64_t* q_empty = q_full + 1;
    uint64_t* item_full = q_full + 2;   // [2]
    uint64_t* item_empty = q_full + 4;  // [2]
    uint64_t* fin = q_full + 6;         // every product has completed
    uint64_t* s_full = q_full + 7;      // [TILES] each
    uint64_t* s_free = s_full + TILES;
    uint64_t* o_empty = s_full + 2 * TILES;
    uint64_t* p_full = s_full + 3 * TILES;   // [TILES][P buffers] each
    uint64_t* pv_done = p_full + PB * TILES;
    G4Item* s_items = reinterpret_cast<G4Item*>(smem + T::kOffItem);
    uint32_t* err = &hdr->error_bits;
    const int G = a.num_q_heads / a.num_kv_heads;
    constexpr int kMma0 = T::kSoft, kQw = T::kSoft + 2, kRawW = T::kSoft + 3, kConv0 = T::kSoft + 4;

    auto init_barriers = [&]() {
        for (int i = 0; i < NK; ++i) {
            mbar_init(&k_full[i], 2);  // (converter warps)
            mbar_init(&k_empty[i], TILES);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(&v_full[i], 2);
            mbar_init(&v_empty[i], TILES);
        }
        for (int i = 0; i < NR; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_empty[i], 4);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, TILES);
        mbar_init(fin, TILES);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&turned[i], 2);
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], T::kThreads / 32);
        }
        for (int t = 0; t < TILES; ++t) {
            mbar_init(&s_full[t], 1);
            mbar_init(&s_free[t], 4);
            mbar_init(&o_empty[t], 4);
            for (int b = 0; b < PB; ++b) {
                mbar_init(&p_full[PB * t + b], 4);
                mbar_init(&pv_done[PB * t + b], 1);
            }
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    };
    if (tid == 0) {
        init_barriers();
        s_abort = 0;
        s_again = -1;
    }
    if (warp == kMma0) tmem_alloc(tmem_slot, T::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // All roles' work on items with V and P in f16, or in bf16. (Two copies of the code: with the types asked for where they
    // matter, the instruction caches hold less of what runs, and 4 x 4096 prompts take 540 to 570 us, not 497.)
    auto work = [&](auto f16) {
        constexpr bool kF16 = decltype(f16)::value;
        uint32_t items = 0;  // items this CTA has taken (ring slots, q phases)
        auto next_item_of = [&](G4Item& it, auto alone) -> bool {
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
        auto next_item = [&](G4Item& it) { return next_item_of(it, std::false_type()); };

        G4Item it;
        if (warp < T::kSoft) {
            // ---------------- softmax and epilogue: thread = row of its tile ----------------
            if constexpr (TILES == 2) g4_regs_inc<T::kRegsSoft>();
            const int t = warp >> 2, quarter = warp & 3;
            const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
            const uint32_t col_s = tmem + lane_off + T::kColS + t * BK, col_p = tmem + lane_off + T::kColP + t * PB * (BK / 2),
                           col_o = tmem + lane_off + T::kColO + t * D;
            [[maybe_unused]] const float cap = a.soft_cap, cap_k2 = cap != 0.f ? 2.f * kLog2e / cap : 0.f;
            const float scale = a.sm_scale / kDown, c_log2 = scale * kLog2e;
            // without a soft cap (and with a positive scale) the maximum is taken on the raw scores and the scale goes into
            // the exponent's multiply-add
            const bool fold = !CAP && c_log2 > 0.f;
            const float cs = fold ? c_log2 : 1.f;
            uint32_t nblk = 0;  // blocks this tile has processed; block n's P lies in buffer n % PB
            auto pv_of = [&](uint32_t n) { return mbar_wait(&pv_done[PB * t + n % PB], (n / PB) & 1, err); };
            bool ok = true;
            while (ok && next_item(it)) {
                const int n_rows = it.q_len * G;
                if (it.row + t * 128 >= n_rows) continue;  // this item has no such tile
                const int R = it.row + t * 128 + quarter * 32 + lane;
                const bool rv = R < n_rows;
                // (a row that is not there sees what the first one does)
                const int qpos = it.kv_len - it.q_len + (rv ? R : it.row) / G;
                const int wlo = a.sliding_window > 0 ? qpos - a.sliding_window + 1 : 0;
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
                    if constexpr (CAP) {
                        // small logits (the warp's every |x * scale| <= |cap| / 4): the series form, on the FMA pipe
                        float am = 0.f;
#pragma unroll
                        for (int i = 0; i < BK; i += 2) am = fmax3(am, fabsf(x[i]), fabsf(x[i + 1]));
                        if (__all_sync(0xffffffffu, am * fabsf(scale) <= 0.25f * fabsf(cap))) {
                            const float ic = 1.f / (cap * kLog2e);
#pragma unroll
                            for (int i = 0; i < BK; i += 2) {
                                const float2 y = soft_cap_small2(fmul2(make_float2(x[i], x[i + 1]), make_float2(c_log2, c_log2)), ic);
                                x[i] = y.x;
                                x[i + 1] = y.y;
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < BK; ++i) x[i] = soft_cap(x[i] * scale, cap, cap_k2) * kLog2e;
                        }
                    } else if (!fold) {
#pragma unroll
                        for (int i = 0; i < BK; ++i) x[i] *= c_log2;
                    }
                    const int lo = wlo - (it.block0 + j) * BK, hi = qpos - (it.block0 + j) * BK;  // columns [lo, hi] are seen
                    if (__any_sync(0xffffffffu, lo > 0 || hi < BK - 1)) {
#pragma unroll
                        for (int i = 0; i < BK; ++i) x[i] = i >= lo && i <= hi ? x[i] : -INFINITY;
                    }
                    float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < BK; i += 2) mx4[(i >> 1) & 3] = fmax3(mx4[(i >> 1) & 3], x[i], x[i + 1]);
                    const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * cs;  // log2 units
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
                        if (!pv_of(nblk - 1)) {  // the previous block's PV has written O
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
                    const float2 cs2 = make_float2(cs, cs), nmu2 = make_float2(nmu + kUpP, nmu + kUpP);
                    // the last PV of this buffer has read it
                    if (nblk >= PB && !pv_of(nblk - PB)) {
                        ok = false;
                        break;
                    }
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
                            if (!kF16) p = fmul2(p, make_float2(kDownV / kDown, kDownV / kDown));
                            pk[e] = kF16 ? pack_f16(p.x, p.y) : pack_bf16(p.x, p.y);
                        }
                        tmem_st16_nowait(col_p + nblk % PB * (BK / 2) + c * 16, pk);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[PB * t + nblk % PB]);
                    l = l * alpha + ((sum2[0].x + sum2[1].x) + (sum2[0].y + sum2[1].y));
                }
                // epilogue: O of the last PV
                if (ok && pv_of(nblk - 1)) {
                    tc_fence_after();
                    const float inv = l > 0.f ? 1.f / (l * kDownV) : 0.f;
                    __nv_bfloat16* dst = a.out + ((size_t)(it.q_start + (rv ? R / G : 0)) * a.num_q_heads + it.head * G + (rv ? R % G : 0)) * D;
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        float o[32];
                        tmem_ld32(col_o + c * 32, o);
                        if (rv) {
                            uint4* d4 = reinterpret_cast<uint4*>(dst + c * 32);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                d4[i] = make_uint4(pack_bf16(o[8 * i] * inv, o[8 * i + 2] * inv), pack_bf16(o[8 * i + 4] * inv, o[8 * i + 6] * inv),
                                                   pack_bf16(o[8 * i + 1] * inv, o[8 * i + 3] * inv), pack_bf16(o[8 * i + 5] * inv, o[8 * i + 7] * inv));
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
            __syncwarp();
            if constexpr (TILES == 2) g4_regs_dec<T::kRegsLaunch>();  // (as it was: what follows is compiled for that)
        } else if (warp < kConv0) {
            if constexpr (TILES == 2) g4_regs_dec<T::kRegsRest>();
            if (warp >= kMma0 && warp < kMma0 + TILES) {
                // ---------------- MMA issuer of tile t (a constant in either branch) ----------------
                // One lane, elected once, does all of it: the ring positions and phases are its registers, and a commit
                // tracks the products of its own thread alone.
                auto issue = [&](auto tile) {
                    constexpr int t = decltype(tile)::value;
                    constexpr uint32_t idesc_qk = umma_idesc_bf16(128, BK, false, false);
                    constexpr uint32_t idesc_pv = umma_idesc_16(128, D, false, true, kF16);
                    const uint64_t qdesc = umma_desc_sw128(smem_u32(smem + t * T::kQTile), 16, 1024);
                    const uint64_t kdesc = umma_desc_sw128(smem_u32(smem + T::kOffK), 16, 1024);
                    const uint64_t vdesc = umma_desc_sw128(smem_u32(smem + T::kOffV), 64 * 128, 1024);
                    const uint32_t col_s = tmem + T::kColS + t * BK, col_p = tmem + T::kColP + t * PB * (BK / 2), col_o = tmem + T::kColO + t * D;
                    uint32_t jk = 0, jv = 0;          // ring positions
                    uint32_t n_own = 0;               // QKs of this tile
                    uint32_t npv = 0, no = 0;         // PVs, and items this tile has had
                    bool ok = true;
                    while (ok && next_item_of(it, std::true_type())) {
                        const int n_rows = it.q_len * G;
                        const bool active = it.row + t * 128 < n_rows;
                        ok = mbar_wait(q_full, (items - 1) & 1, err);
                        for (int j = 0; ok && j <= it.blocks; ++j) {
                            if (j < it.blocks) {  // QK of block j
                                const uint32_t slot = jk % NK;
                                ok = mbar_wait(&k_full[slot], (jk / NK) & 1, err);
                                ++jk;
                                if (active) {
                                    // the scores that lie there have been read
                                    if (n_own > 0) ok = ok && mbar_wait(&s_free[t], (n_own - 1) & 1, err);
                                    if (!ok) break;
                                    tc_fence_after();
                                    const uint64_t kb = kdesc + (uint64_t)((slot * T::kTile) >> 4);
#pragma unroll
                                    for (int ks = 0; ks < D / 16; ++ks)
                                        umma_bf16(col_s, qdesc + (((ks >> 2) * T::kQPanel + (ks & 3) * 32) >> 4),
                                                  kb + (((ks >> 2) * T::kPanel + (ks & 3) * 32) >> 4), idesc_qk, ks > 0 ? 1u : 0u);
                                    umma_commit(&s_full[t]);
                                    umma_commit(&k_empty[slot]);
                                    if (j + 1 == it.blocks) umma_commit(q_empty);
                                    ++n_own;
                                } else {
                                    if (!ok) break;
                                    mbar_arrive(&k_empty[slot]);
                                    if (j + 1 == it.blocks) mbar_arrive(q_empty);
                                }
                            }
                            if (j > 0) {  // PV of block j - 1
                                const uint32_t pb = npv % PB, slot = jv % NV;
                                if (active) {
                                    if (j == 1 && no > 0) ok = ok && mbar_wait(&o_empty[t], (no - 1) & 1, err);
                                    ok = ok && mbar_wait(&p_full[PB * t + pb], (npv / PB) & 1, err);
                                }
                                ok = ok && mbar_wait(&v_full[slot], (jv / NV) & 1, err);
                                if (!ok) break;
                                ++jv;
                                if (active) {
                                    const uint64_t vb = vdesc + (uint64_t)((slot * T::kTile) >> 4);
                                    tc_fence_after();
#pragma unroll
                                    for (int kk = 0; kk < BK / 16; ++kk)
                                        umma_bf16_ta(col_o, col_p + pb * (BK / 2) + kk * 8, vb + ((kk * 16 * 128) >> 4), idesc_pv,
                                                     (j > 1 || kk > 0) ? 1u : 0u);
                                    umma_commit(&v_empty[slot]);
                                    umma_commit(&pv_done[PB * t + pb]);
                                    ++npv;
                                } else {
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
            } else if (warp == kQw) {
                // ---------------- items and Q ----------------
                const int n_items = hdr->num_items[1];
                uint32_t fetched = 0;
                // Items with a V that f16 does not fit are done again in bf16 once there are no more: a chain through the list's
                // entries (an item's type follows from its values alone, not from which CTA took it when).
                auto ask = [&](uint32_t n) {
                    if (!kF16 || s_abort) return;
                    if (!mbar_wait(&turned[n & 1], (n >> 1) & 1, err)) {
                        s_abort = 1;
                    } else if (!item_fits[2 * (n & 1)] || !item_fits[2 * (n & 1) + 1]) {
                        a.pre_items[s_items[n & 1].place].key_begin = s_again;
                        s_again = s_items[n & 1].place;
                    }
                };
                auto fetch = [&]() {
                    const uint32_t slot = fetched & 1, ph = (fetched >> 1) & 1;
                    G4Item n;
                    n.seq = -1;
                    if (!mbar_wait(&item_empty[slot], ph ^ 1, err)) s_abort = 1;
                    // beside decode, no new item once most decode CTAs with a share are out of work: what is left goes to
                    // the launch after decode, on every SM
                    const bool stop = s_abort || (kF16 && !tail && a.overlap && hdr->dec_ctas > 0 &&
                                                  *(volatile const int*)&hdr->next_item[0] >= max(1, hdr->dec_ctas * kPrefillStopPercent / 100));
                    if (fetched >= 2) ask(fetched - 2);
                    int place = n_items;
                    if (kF16 && !stop) place = atomicAdd(&hdr->next_item[1], 1);
                    if (!kF16 && !s_abort && s_again >= 0) {
                        place = s_again;
                        s_again = a.pre_items[place].key_begin;
                    }
                    if (place < n_items) {
                        const WorkItem w = a.pre_items[place];
                        n.place = place;
                        n.seq = w.seq;
                        n.head = w.head;
                        n.row = w.row_begin;
                        n.q_start = a.cu_q_lens[w.seq];
                        n.q_len = a.cu_q_lens[w.seq + 1] - n.q_start;
                        n.kv_len = a.kv_lens[w.seq];
                        const int last = min(n.row + 128 * TILES, n.q_len * G) - 1;
                        const int qmin = n.kv_len - n.q_len + n.row / G, qmax = n.kv_len - n.q_len + last / G;
                        n.block0 = a.sliding_window > 0 ? max(0, qmin - a.sliding_window + 1) / BK : 0;
                        n.blocks = qmax / BK + 1 - n.block0;
                    } else if (fetched >= 1) {
                        ask(fetched - 1);  // (no more items)
                    }
                    s_items[slot] = n;
                    mbar_arrive(&item_full[slot]);
                    ++fetched;
                };
                bool ok = true;
                if (lane == 0) fetch();
                __syncwarp();
                while (ok && next_item(it)) {
                    ok = mbar_wait(q_empty, items & 1, err);  // the previous item's last QK
                    if (!ok) break;
                    const int n_rows = it.q_len * G, tiles = min(TILES, cdiv(n_rows - it.row, 128));
                    if (q_tma) {
                        if (lane == 0) {
                            mbar_arrive_expect_tx(q_full, tiles * T::kQTile);
                            for (int t = 0; t < tiles; ++t)
#pragma unroll
                                for (int p = 0; p < T::DP; ++p)
                                    tma_load_3d(smem_u32(smem + t * T::kQTile + p * T::kQPanel), &tm_q, 64 * p, it.head * G,
                                                it.q_start + (it.row + t * 128) / G, q_full);
                        }
                    } else {
                        // a group size that does not divide a tile: 16 bytes at a time, rows that are not there as zeros
                        for (int i = lane; i < tiles * 128 * (D / 8); i += 32) {
                            const int r = i / (D / 8), c = i % (D / 8), R = it.row + r, t = r >> 7, tr = r & 127;
                            const bool rv = R < n_rows;
                            cp_async16(smem_u32(smem + t * T::kQTile + (c >> 3) * T::kQPanel + tr * 128 + (((c & 7) ^ (tr & 7)) << 4)),
                                       a.q + ((size_t)(it.q_start + (rv ? R / G : 0)) * a.num_q_heads + it.head * G + (rv ? R % G : 0)) * D + c * 8, rv);
                        }
                        cp_async_commit();
                        cp_async_wait<0>();
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(q_full);
                    }
                    if (lane == 0) fetch();
                    __syncwarp();
                }
                if (!ok) s_abort = 1;
                if (lane == 0 && s_abort) {
                    // an aborted warp still ends the other warps' wait for an item; a copy under way lands (bounded)
                    if (!ok) fetch();
                    if (items > 0) mbar_wait(q_full, (items - 1) & 1, err);
                }
                __syncwarp();
            } else if (warp == kRawW) {
                // ---------------- raw rows: a tensor copy a page (or a block's part of one) of this head's rows ----------------
                // (page sizes no box tiles a block with: 16 bytes at a time)
                const uint8_t* kv = static_cast<const uint8_t*>(a.kv_pages);
                const size_t slot_bytes = (size_t)a.num_kv_heads * F::kRow;
                const int lbr = __ffs(box_rows) - 1, lps = __ffs(a.page_size) - 1;
                uint32_t jr = 0;
                bool ok = true;
                while (ok && next_item(it)) {
                    const int* tbl = a.page_indices + (size_t)it.seq * a.pages_per_seq;
                    const int ke = g4_key_end(it, G, TILES);
                    auto page_of = [&](int j) -> int {
                        const int key = (it.block0 + j) * BK + lane * box_rows;
                        return box_rows && lane * box_rows < BK && j < it.blocks && key < ke ? __ldg(tbl + (key >> lps)) : 0;
                    };
                    int page_next = page_of(0);
                    for (int j = 0; ok && j < it.blocks; ++j, ++jr) {
                        int page = page_next;
                        page_next = page_of(j + 1);
                        const int key0 = (it.block0 + j) * BK, valid = min(BK, ke - key0);
                        const uint32_t slot = jr % NR, ph = (jr / NR) & 1, dst = smem_u32(smem + T::kOffRaw + slot * T::kRaw);
                        ok = mbar_wait(&raw_empty[slot], ph ^ 1, err);
                        if (!ok) break;  // (every lane has waited)
                        if (box_rows) {
                            const int boxes = (valid + box_rows - 1) >> lbr;
                            if (lane < boxes && (unsigned)page >= (unsigned)a.total_num_pages) {
                                set_error(err, RPA_DEV_ERR_PAGE);
                                page = 0;  // an in-bounds page keeps the barrier's byte count; the error is recorded
                            }
                            if (lane == 0) mbar_arrive_expect_tx(&raw_full[slot], (uint32_t)(boxes * box_rows * F::kRow));
                            __syncwarp();
                            if (lane < boxes)
                                tma_load_3d(dst + lane * box_rows * F::kRow, &tm_kv, 0, (page << lps) + ((key0 + lane * box_rows) & (a.page_size - 1)), it.head,
                                            &raw_full[slot]);
                        } else {
                            for (int i = lane; i < valid * (F::kRow / 16); i += 32) {
                                const int r = i / (F::kRow / 16), c = i % (F::kRow / 16), key = key0 + r;
                                int p = __ldg(tbl + key / a.page_size);
                                if ((unsigned)p >= (unsigned)a.total_num_pages) {
                                    set_error(err, RPA_DEV_ERR_PAGE);
                                    p = 0;
                                }
                                cp_async16(dst + r * F::kRow + c * 16,
                                           kv + ((size_t)p * a.page_size + key % a.page_size) * slot_bytes + (size_t)it.head * F::kRow + c * 16, true);
                            }
                            cp_async_commit();
                            cp_async_wait<0>();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&raw_full[slot]);
                        }
                    }
                    if (!ok) s_abort = 1;
                }
                if (lane == 0 && s_abort)  // copies under way land (bounded) before shared memory goes
                    for (uint32_t i = jr > NR ? jr - NR : 0; i < jr; ++i) mbar_wait(&raw_full[i % NR], (i / NR) & 1, err);
                __syncwarp();
            } else {
                while (next_item(it)) {
                }
            }
            __syncwarp();
            if constexpr (TILES == 2) g4_regs_inc<T::kRegsLaunch>();
        } else {
            if constexpr (TILES == 2) g4_regs_dec<T::kRegsRest>();
            // ---------------- converters: a row of a block a thread ----------------
            constexpr int CH = D / 32;  // 16-byte chunks of numbers a row
            const int row = (tid - kConv0 * 32) & 63, part = warp >= kConv0 + 2;
            const uint32_t off = smem_u32(smem + T::kOffRaw) + row * F::kRow + part * F::kPart;
            const uint32_t off_sm = smem_u32(smem + T::kOffRaw) + row * F::kRow + F::kParams + part * 4 * F::NG;
            const uint32_t panel = smem_u32(smem + (part ? T::kOffV : T::kOffK) + row * 128);
            uint64_t *full = part ? v_full : k_full, *empty = part ? v_empty : k_empty;
            const uint32_t depth = part ? NV : NK;
            uint32_t jb = 0;  // blocks
            bool ok = true;
            while (ok && next_item(it)) {
                bool fits = true;
                // keys that some row of the item sees: [k0, ke); the others are zeros, whatever lies there
                const int ke = g4_key_end(it, G, TILES);
                const int k0 = g4_key_begin(it, G, a.sliding_window);
                int key = it.block0 * BK + row;
#pragma unroll 1
                for (int j = 0; ok && j < it.blocks; ++j, ++jb, key += BK) {
                    const uint32_t raw = jb % NR, slot = jb % depth, src = raw * T::kRaw;
                    ok = mbar_wait(&raw_full[raw], (jb / NR) & 1, err);
                    const bool in = key < ke && key >= k0;
                    if (kF16 && part) {  // (before the wait for a free panel)
#pragma unroll
                        for (int g = 0; g < F::NG; ++g) fits = fits && (!in || g4_fits_f16(lds32(off_sm + src + 4 * g)));
                    }
                    ok = ok && mbar_wait(&empty[slot], ((jb / depth) & 1) ^ 1, err);
                    if (!ok) break;
                    const uint32_t stage = panel + slot * T::kTile;
                    // A chunk's numbers and scales are loaded while the one before is turned. The loop stays rolled: unrolled
                    // over a block, this code and the softmax's, each run through once a block, come too slowly from the
                    // instruction caches (4 x 4096 prompts 878 us).
                    auto turn = [&](auto kind) {
                        constexpr bool kV = decltype(kind)::value, kHalf = kV && kF16;
                        uint4 w = lds128(off + src);
                        uint32_t sm = lds32(off_sm + src);
#pragma unroll 1
                        for (int c = 0; c < CH; ++c) {
                            if (!in) sm = 0u;
                            const uint32_t p = kHalf ? pack_f16(bf16_lo(sm) * (kDownV * 0x1p24f), bf16_hi(sm) * kDownV)
                                                           : bf16x2_mul(sm, 0x25006780u);  // (s 2^80, m 2^-53)
                            const uint32_t s2 = __byte_perm(p, p, 0x1010), m2 = __byte_perm(p, p, 0x3232);
                            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
                            const int next = c + 1 < CH ? c + 1 : 0;
                            w = lds128(off + src + next * 16);
                            sm = lds32(off_sm + src + 4 * (next * 32 / F::kGroup));
                            const uint32_t s2_16 = kHalf ? f16x2_fma(s2, 0x2c002c00u, 0u) : bf16x2_mul(s2, 0x3d803d80u);  // a 16th
                            uint4 x[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                x[e] = !kV     ? g4_panel8(ww[e], s2, m2)
                                       : kHalf ? g4_panel8_v_f16(ww[e], s2, s2_16, m2)
                                               : g4_panel8_v(ww[e], s2, s2_16, m2);
                            // 16-byte chunks 4 c .. 4 c + 3 of the row: half of a panel's 128 bytes
                            const uint32_t to = stage + (c >> 1) * T::kPanel, low = (c & 1) << 2;
#pragma unroll
                            for (int e = 0; e < 4; ++e) sts128(to + (((low + e) ^ (row & 7)) << 4), x[e]);
                        }
                    };
                    if (part)
                        turn(std::true_type());
                    else
                        turn(std::false_type());
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&full[slot]);
                        mbar_arrive(&raw_empty[raw]);
                    }
                }
                if (kF16 && part) {
                    fits = __all_sync(0xffffffffu, fits);
                    if (lane == 0) {
                        item_fits[2 * ((items - 1) & 1) + warp - kConv0 - 2] = fits;
                        mbar_arrive(&turned[(items - 1) & 1]);
                    }
                }
                if (!ok) s_abort = 1;
            }
            __syncwarp();
            if constexpr (TILES == 2) g4_regs_inc<T::kRegsLaunch>();
        }
    };
    work(std::true_type());
    tc_fence_before();
    __syncthreads();  // (every role has ended, and with it every copy and product)
    tc_fence_after();
    if (s_again >= 0 && !s_abort) {
        __syncthreads();
        if (tid == 0) {
            for (int i = 0; i < T::kBars; ++i) mbar_inval(&k_full[i]);
            init_barriers();
        }
        __syncthreads();
        work(std::false_type());
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }
    if (warp == kMma0) tmem_dealloc(tmem, T::kTmemCols);
}

// Rows of `bytes` bytes (a multiple of 16, at most 1024), [tokens][heads] of them, dense, as a tensor [heads][tokens][row]
// with a box of b_heads x b_tokens rows, each `pitch` bytes apart where it lands (zeros behind the row), without a swizzle.
bool make_tmap_heads(CUtensorMap* tm, const void* base, uint64_t bytes, uint64_t heads, uint64_t tokens, uint32_t pitch, uint32_t b_tokens,
                     uint32_t b_heads) {
    static PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    if (!enc) {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return false;
        enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }
    const cuuint64_t dims[3] = {bytes / 4, tokens, heads};
    const cuuint64_t strides[2] = {bytes * heads, bytes};
    const cuuint32_t box[3] = {pitch / 4, b_tokens, b_heads};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool CAP>
static cudaError_t launch_pre(const RpaArgs& a, int num_sms, cudaStream_t stream, int tail) {
    using T = G4Pre<D>;
    auto kern = g4_prefill_kernel<D, CAP>;
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
        if (T::TILES == 2 && fa.numRegs != T::kRegsLaunch) return cudaErrorLaunchOutOfResources;
        configured[dev] = true;
    }
    CUtensorMap tq, tkv;
    memset(&tq, 0, sizeof tq);
    memset(&tkv, 0, sizeof tkv);
    const int G = a.num_q_heads / a.num_kv_heads, ps = a.page_size;
    const int q_tma = 128 % G == 0 && make_tmap_bf16(&tq, a.q, D, a.num_q_heads, a.max_num_tokens, G, 128 / G);
    // boxes of a page's rows, or a block's part of them: at least 8, so that each starts on 128 bytes
    int box_rows = (ps & (ps - 1)) == 0 && ps >= 8 ? (ps < T::BK ? ps : T::BK) : 0;
    if ((long long)a.total_num_pages * ps > INT32_MAX) box_rows = 0;
    if (box_rows && !make_tmap_heads(&tkv, a.kv_pages, G4<D>::kRow, a.num_kv_heads, (uint64_t)a.total_num_pages * ps, G4<D>::kRow, box_rows, 1)) box_rows = 0;
    ProfScope prof(tail == 1 ? "rpa_g4_prefill_tail" : "rpa_g4_prefill", stream);
    return launch_pdl(kern, dim3(num_sms), dim3(T::kThreads), T::kSmem, stream, a.overlap && !tail, a, tq, tkv, q_tma, box_rows, tail);
}

cudaError_t launch_g4_prefill(const RpaArgs& a, int num_sms, cudaStream_t stream, int tail) {
    const bool cap = a.soft_cap != 0.f;
    switch (a.head_dim) {
        case 64: return cap ? launch_pre<64, true>(a, num_sms, stream, tail) : launch_pre<64, false>(a, num_sms, stream, tail);
        case 128: return cap ? launch_pre<128, true>(a, num_sms, stream, tail) : launch_pre<128, false>(a, num_sms, stream, tail);
        case 256: return cap ? launch_pre<256, true>(a, num_sms, stream, tail) : launch_pre<256, false>(a, num_sms, stream, tail);
        default: return cudaErrorInvalidValue;
    }
}

int g4_prefill_rows(int head_dim) { return head_dim == 256 ? 128 : 256; }

}  // namespace rpa
