// Decode-class attention over the 4-bit cache (rpa_g4_forward: sequences of at most 16 query rows a KV head), for
// sm_103a.
//
//   S = c (s (Q.n) + m sum Q) per group of K,   O = sum_k p_k (s_k n_k + m_k) per group of V.
//
// A key costs 1.125 bytes an element of K and V together (D = 128: 144 a head), so the work a byte is four times that
// of a bf16 cache: what bounds the kernel is issue slots beside HBM.  So nothing is converted.  The numbers
// go to the tensor cores as they lie: with all other bits of a half masked away, n is the bf16 subnormal n 2^-133
// (bits 0-3) or n 2^-129 (bits 4-7: subnormals and the lowest exponent share one step), which mma.sync multiplies
// exactly (checked: A = n 2^-133 and n 2^-129 against B = 2^100).  One word of 8 numbers gives four operand
// registers with four ANDs and a shift.  The scales are applied to the results:
//   * K: a k-step's 16 dims are of one group, so each group has an accumulator of its own; S takes s and m of
//     its key from one 16-byte load a key, and sum Q of the group from registers.  Q is brought to 2^119..2^120
//     by a power of two of its row (its other bf16 bits stay).  Every product is exact.
//   * V: P s goes in as the B operand, one a group; what m adds is a sum over keys of p (m + 7.5 s) in float32,
//     less 7.5 times the sum of the rounded P s, which a product with ones gives: the rounding of P s to bf16 (2^-8
//     of itself) then counts for n - 7.5, a value's distance from the middle, not for n.
// Otherwise as the kernel for wider caches: a producer warp resolves pages two stages ahead and copies 16 keys' rows of HG
// heads in one tensor copy (page sizes that are powers of two from 16 on; else a row of a head in one bulk copy: 128
// decodes over up to 8192 keys 193 us, not 165); a consumer warp a KV head, keys on the M side of m16n8k16, up to 8 query
// rows on its N side; items split the keys (flash-decoding) along the plan's equal shares, and a group's last CTA
// joins its pieces.
//
// 128 decodes over 512 to 8192 keys, 32/8 heads of 128 (605 MB): 165 us, 3.7 TB/s, of heads of 64 113 us. The copies alone
// take 155 us, the arithmetic alone 158: 12 warps an SM that compute issue in 47 % of the cycles, each mostly waiting
// on its own chain of loads, products and exponentials, and boxes of 144-byte rows 1152 bytes apart bring HBM to half its
// rate. (All 8 heads of such a row in one copy: 135 us for the copies, but 8 + 1 warps a CTA have 96 registers each and spill:
// 170 us; with the copies asked for by the last warp through a stage, no producer, 128 registers, and no spills: 165
// us, and 28 us instead of 24 for 5 decodes.)
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "g4.cuh"
#include "kernels.h"
#include "profile.h"

namespace rpa {

template <int D, int HG>
struct G4Dec {
    static constexpr int BK = 2 * kDecodeBK;             // keys a stage: two tiles of 16
    // tiles at once: two, so that the chains of loads, products, maxima and exponentials of one run beside the other's (and
    // the maximum's exchange and the barriers come once for both); head_dim 256 has no registers for that
    static constexpr int NT = D == 256 ? 1 : 2;
    // A stage is two tiles, a tile its heads one behind another, each 16 rows of kPitch bytes. Rows 8 or 24 words apart modulo the 32 banks
    // let K's 8-byte loads (four rows of 32 bytes a half-warp) and, with the keys' order of key_of, V's 4-byte loads
    // touch every bank once; at head_dim 64 (4- and 2-byte loads) 20 words do. A box copies the padding with its rows.
    static constexpr int kPitch = D == 128 ? 160 : G4<D>::kRow;
    static constexpr int kHead = 16 * kPitch, kTile = HG * kHead, kStage = 2 * kTile;
    static constexpr int STAGES = 3;
    static constexpr int kBarOff = STAGES * kStage;
    static constexpr int kSmem = kBarOff + 2 * STAGES * 8;
    static constexpr int kThreads = (HG + 1) * 32;
    static constexpr int kCtas = D == 256 ? 2 : 3;  // an SM's: as many as the stages let in
};

// The stage's key in row r of the M side (and r + 8 the one 8 further on): the order in which both K's and V's rows
// lie apart in the banks.
__device__ __forceinline__ int g4_key_of(int r) { return r ^ ((r >> 2) & 1); }

template <int D, int HG>
__global__ void __launch_bounds__(G4Dec<D, HG>::kThreads, G4Dec<D, HG>::kCtas)
    g4_decode_kernel(const __grid_constant__ RpaArgs a, const __grid_constant__ CUtensorMap tm_kv, int boxes) {
    using T = G4Dec<D, HG>;
    using F = G4<D>;
    constexpr int BK = T::BK, STAGES = T::STAGES, NG = F::NG;
    constexpr int KW = F::kGroup / 32;       // a lane's words of a group's K row (8 dims each): 1 or 2
    constexpr int TG = F::kGroup / 16;       // V tiles of 16 dims a group: 2 or 4
    constexpr int kRowO = HG * kDecodeRows;  // rows of an item's partial result
    constexpr float kUp = 0x1p69f;           // 2^(133 - 64): P s goes in times 2^64
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + T::kBarOff);
    uint64_t* empty = full + STAGES;
    __shared__ WorkItem s_item;
    __shared__ int s_item_idx, s_last;
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool producer = warp == HG;
    WsHeader* hdr = a.hdr;
    uint32_t* err = &hdr->error_bits;
    const int Hkv = a.num_kv_heads, G = a.num_q_heads / Hkv;
    const uint8_t* kv = static_cast<const uint8_t*>(a.kv_pages);

    // zero the stages once: rows that are never copied (slots past the keys) stay finite
    for (int i = tid * 16; i < STAGES * T::kStage; i += blockDim.x * 16) *reinterpret_cast<uint4*>(smem + i) = make_uint4(0, 0, 0, 0);
    if (tid == 0) {
        for (int st = 0; st < STAGES; ++st) {
            mbar_init(&full[st], 1);
            mbar_init(&empty[st], HG);
        }
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    fence_proxy_async_smem();
    __syncthreads();
    uint32_t pipe = 0;                                  // blocks this CTA has pushed through the ring so far
    uint32_t issued = 0;                                // producer's first lane: blocks it has asked for

    // prefill first (the plan gave it every SM): start once it has ended (no-op on an ordinary launch)
    if (hdr->prefill_ctas >= a.num_sms && hdr->num_items[1] > 0) pdl_wait();
    const int n_items = hdr->num_items[0], n_static = hdr->dec_ctas, n_shares = hdr->dec_shares;
    int my_it = 0, my_end = 0;
    bool pool_left = true;
    if (tid == 0 && (int)blockIdx.x < n_static) {
        my_it = min(max(a.cta_first[blockIdx.x], 0), n_items);
        my_end = min(max(a.cta_first[blockIdx.x + 1], my_it), n_items);
    }
    while (true) {
        if (tid == 0) {
            while (my_it >= my_end && pool_left) {
                const int c = n_static + atomicAdd(&hdr->next_item[2], 1);
                if (c >= n_shares) {
                    pool_left = false;
                } else {
                    my_it = min(max(a.cta_first[c], 0), n_items);
                    my_end = min(max(a.cta_first[c + 1], my_it), n_items);
                }
            }
            const int it = my_it < my_end ? my_it++ : -1;
            s_item.seq = -1;
            s_item_idx = it;
            if (it >= 0) s_item = a.dec_items[it];
        }
        __syncthreads();
        const WorkItem w = s_item;
        const int self = s_item_idx;
        if (w.seq < 0 || s_abort) break;
        const int s = w.seq, q_start = a.cu_q_lens[s], q_len = a.cu_q_lens[s + 1] - q_start, kv_len = a.kv_lens[s];
        const int n_rows = q_len * G, kb = w.key_begin, ke = w.key_end, n_blocks = ke > kb ? cdiv(ke - kb, BK) : 0;
        const int h0 = w.head, seg_heads = min(HG, Hkv - h0);
        const uint32_t seg_bytes = seg_heads * F::kRow;

        if (producer) {
            // Pages are looked up two stages ahead (one was not enough: a stage then took a load's latency).
            const int* tbl = a.page_indices + (size_t)s * a.pages_per_seq;
            // A lane asks for a tile's keys of all its heads with one box (page sizes that are whole tiles; the keys begin at a
            // multiple of 16, so that a tile lies in one page), or for one key, head by head.
            const int rows = boxes ? 16 : 1, lps = __ffs(a.page_size) - 1;
            auto page_of = [&](int blk) -> int {
                const int key = kb + blk * BK + lane * rows;
                return blk < n_blocks && lane * rows < BK && key < ke ? __ldg(tbl + (boxes ? key >> lps : key / a.page_size)) : -1;
            };
            int page_next = page_of(0), page_then = page_of(1);
            for (int blk = 0; blk < n_blocks; ++blk) {
                const uint32_t q = pipe + blk, st = q % STAGES, ph = (q / STAGES) & 1;
                const int page = page_next;
                page_next = page_then;
                page_then = page_of(blk + 2);
                const int key = kb + blk * BK + lane * rows;
                const bool want = lane * rows < BK && key < ke, ok = want && (unsigned)page < (unsigned)a.total_num_pages;
                if (want && !ok) set_error(err, RPA_DEV_ERR_PAGE);
                const uint32_t mask = __ballot_sync(0xffffffffu, ok);
                int go = 1;
                if (lane == 0) {
                    go = mbar_wait(&empty[st], ph ^ 1, err);
                    if (go) {
                        mbar_arrive_expect_tx(&full[st], __popc(mask) * (boxes ? (uint32_t)T::kTile : (uint32_t)(seg_heads * F::kRow)));
                        issued = q + 1;
                    } else {
                        s_abort = 1;
                    }
                }
                go = __shfl_sync(0xffffffffu, go, 0);
                if (!go) break;
                if (ok) {
                    const uint32_t dst = smem_u32(smem + st * T::kStage);
                    if (boxes) {
                        tma_load_3d(dst + lane * T::kTile, &tm_kv, 0, (page << lps) + (key & (a.page_size - 1)), h0, &full[st]);
                    } else {
                        const uint8_t* src = kv + (((size_t)page * a.page_size + key % a.page_size) * Hkv + h0) * F::kRow;
                        for (int h = 0; h < seg_heads; ++h)
                            bulk_g2s(dst + (lane >> 4) * T::kTile + h * T::kHead + (lane & 15) * T::kPitch, src + h * F::kRow, F::kRow, &full[st]);
                    }
                }
            }
        } else {
            // ---------------- consumer warp: KV head h0 + warp ----------------
            const bool head_ok = warp < seg_heads;
            const int head = h0 + warp, g8 = lane >> 2, q4 = lane & 3, rb = w.row_begin;
            int qpos[2], wlo[2];
            bool rv[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int R = rb + 2 * q4 + j;
                rv[j] = head_ok && R < n_rows;
                qpos[j] = rv[j] ? query_pos(a, q_len, kv_len, R / G) : -1;
                wlo[j] = a.sliding_window > 0 ? qpos[j] - a.sliding_window + 1 : 0;
            }
            // blocks in [all_lo, all_hi] are seen by every row of the item
            const int rl = min(n_rows, rb + kDecodeRows) - 1;
            const int all_hi = min(query_pos(a, q_len, kv_len, rb / G), ke - 1);
            const int all_lo = a.sliding_window > 0 ? query_pos(a, q_len, kv_len, rl / G) - a.sliding_window + 1 : 0;
            // Q^T as B fragments: column g8; word `wd` of group g holds this lane's 8 dims from g * kGroup + q4 *
            // (kGroup / 4) + 8 wd on, and a k-step takes dims (0, 4 | 1, 5) or (2, 6 | 3, 7) of them, as K's masked
            // words come; the second pair of either lies 4 bits higher there, so it is a 16th here
            uint32_t qb[NG * KW * 2][2];
            float qsum[NG][2], to_log2[2];
            {
                const int Rb = rb + g8;
                const bool rvb = head_ok && Rb < n_rows;
                const uint4* qrow = reinterpret_cast<const uint4*>(
                    a.q + ((size_t)(q_start + (rvb ? Rb / G : 0)) * a.num_q_heads + head * G + (rvb ? Rb % G : 0)) * D);
                uint4 raw[NG * KW];
                float mabs = 0.f, sum[NG];
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    sum[g] = 0.f;
#pragma unroll
                    for (int wd = 0; wd < KW; ++wd) {
                        const uint4 v = rvb ? __ldg(qrow + (g * F::kGroup + q4 * (F::kGroup / 4)) / 8 + wd) : make_uint4(0, 0, 0, 0);
                        raw[g * KW + wd] = v;
                        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            sum[g] += bf16_lo(x[e]) + bf16_hi(x[e]);
                            mabs = fmax3(mabs, fabsf(bf16_lo(x[e])), fabsf(bf16_hi(x[e])));
                        }
                    }
                    sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
                    sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
                }
                mabs = fmaxf(mabs, __shfl_xor_sync(0xffffffffu, mabs, 1));
                mabs = fmaxf(mabs, __shfl_xor_sync(0xffffffffu, mabs, 2));
                int ex = 0;
                frexpf(mabs, &ex);                          // mabs < 2^ex
                const int k = max(6, min(120, 120 - ex));   // mabs 2^k in [2^119, 2^120), as far as 2^(133 - k) is a float
                const float qs = ldexpf(1.f, k), rowmul = ldexpf(1.f, 133 - k);
                auto scaled = [&](uint32_t lo, uint32_t hi, float f) {
                    return pack_bf16(fminf(fmaxf(__uint_as_float(lo) * f, -0x1p126f), 0x1p126f),
                                     fminf(fmaxf(__uint_as_float(hi) * f, -0x1p126f), 0x1p126f));
                };
#pragma unroll
                for (int i = 0; i < NG * KW; ++i) {
                    const uint4 v = raw[i];
                    qb[2 * i][0] = scaled(v.x << 16, v.z << 16, qs);                                    // dims 0, 4
                    qb[2 * i][1] = scaled(v.x & 0xffff0000u, v.z & 0xffff0000u, qs * 0.0625f);          // 1, 5
                    qb[2 * i + 1][0] = scaled(v.y << 16, v.w << 16, qs);                                // 2, 6
                    qb[2 * i + 1][1] = scaled(v.y & 0xffff0000u, v.w & 0xffff0000u, qs * 0.0625f);      // 3, 7
                }
                // scores are in units of the products, 2^(k - 133) of their size, until the factor to log2 units
                const float unit = ldexpf(1.f, k - 133);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    to_log2[j] = __shfl_sync(0xffffffffu, rowmul, (2 * q4 + j) * 4) * (a.soft_cap != 0.f ? a.sm_scale : a.sm_scale * kLog2e);
#pragma unroll
                    for (int g = 0; g < NG; ++g) qsum[g][j] = __shfl_sync(0xffffffffu, sum[g] * unit, (2 * q4 + j) * 4);
                }
            }
            // O^T tiles: tile t of group g has this lane's dims g * kGroup + g8 * (kGroup / 8) + 2 t (C rows g8) and
            // + 1 (rows g8 + 8, 4 bits higher), columns (query rows) 2 q4, 2 q4 + 1; psum: the sums of P s
            float o[NG * TG][4], psum[NG][4], mid[NG][2];
#pragma unroll
            for (int i = 0; i < NG * TG; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll
            for (int g = 0; g < NG; ++g) psum[g][0] = psum[g][1] = psum[g][2] = psum[g][3] = mid[g][0] = mid[g][1] = 0.f;
            float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
            const float cap = a.soft_cap, cap_k2 = cap != 0.f ? 2.f * kLog2e / cap : 0.f;
            const int kk = g4_key_of(g8);

            for (int blk = 0; blk < n_blocks; ++blk) {
                const uint32_t qn = pipe + blk, st = qn % STAGES, ph = (qn / STAGES) & 1;
                if (!mbar_wait(&full[st], ph, err)) {
                    s_abort = 1;
                    break;
                }
                if (head_ok) {
#pragma unroll
                    for (int sub = 0; sub < 2; sub += T::NT) {
                        constexpr int NT = T::NT;
                        const int b0 = kb + blk * BK + 16 * sub;  // the tiles' first key
                        if (NT == 1 && b0 >= ke) break;
                        const uint8_t* stg = smem + st * T::kStage + sub * T::kTile + warp * T::kHead;
                        const uint8_t* r0 = stg + kk * T::kPitch;  // this lane's keys: kk and kk + 8 of a tile
                        float sc[NT][4];
                        uint32_t vs[NT][2][NG];  // (s, m) of V's groups
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const uint8_t* rt = r0 + t * T::kTile;
                            uint32_t ks[2][NG];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint4* p = reinterpret_cast<const uint4*>(rt + 8 * h * T::kPitch + F::kParams);
                                if constexpr (NG == 2) {
                                    const uint4 v = p[0];
                                    ks[h][0] = v.x; ks[h][1] = v.y; vs[t][h][0] = v.z; vs[t][h][1] = v.w;
                                } else {
                                    const uint4 u = p[0], v = p[1];
                                    ks[h][0] = u.x; ks[h][1] = u.y; ks[h][2] = u.z; ks[h][3] = u.w;
                                    vs[t][h][0] = v.x; vs[t][h][1] = v.y; vs[t][h][2] = v.z; vs[t][h][3] = v.w;
                                }
                            }
                            // S^T [16 keys x 8 rows], a group at a time
                            sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.f;
#pragma unroll
                            for (int g = 0; g < NG; ++g) {
                                uint32_t x0[KW], x1[KW];
                                const uint8_t* at = rt + g * (F::kGroup / 2) + q4 * (F::kGroup / 8);
                                if constexpr (KW == 2) {
                                    const uint2 u = *reinterpret_cast<const uint2*>(at), v = *reinterpret_cast<const uint2*>(at + 8 * T::kPitch);
                                    x0[0] = u.x; x0[1] = u.y; x1[0] = v.x; x1[1] = v.y;
                                } else {
                                    x0[0] = *reinterpret_cast<const uint32_t*>(at);
                                    x1[0] = *reinterpret_cast<const uint32_t*>(at + 8 * T::kPitch);
                                }
                                float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                                for (int wd = 0; wd < KW; ++wd) {
                                    const uint32_t u = x0[wd], v = x1[wd], u8 = u >> 8, v8 = v >> 8;
                                    const uint32_t f0[4] = {u & 0x000f000fu, v & 0x000f000fu, u & 0x00f000f0u, v & 0x00f000f0u};
                                    const uint32_t f1[4] = {u8 & 0x000f000fu, v8 & 0x000f000fu, u8 & 0x00f000f0u, v8 & 0x00f000f0u};
                                    mma_bf16(acc, f0, qb[2 * (g * KW + wd)][0], qb[2 * (g * KW + wd)][1]);
                                    mma_bf16(acc, f1, qb[2 * (g * KW + wd) + 1][0], qb[2 * (g * KW + wd) + 1][1]);
                                }
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    sc[t][e] = fmaf(bf16_lo(ks[e >> 1][g]), acc[e], fmaf(bf16_hi(ks[e >> 1][g]), qsum[g][e & 1], sc[t][e]));
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) sc[t][e] *= to_log2[e & 1];
                        }
                        if (cap != 0.f) {
#pragma unroll
                            for (int t = 0; t < NT; ++t)
#pragma unroll
                                for (int e = 0; e < 4; ++e) sc[t][e] = soft_cap(sc[t][e], cap, cap_k2) * kLog2e;
                        }
                        if (b0 < all_lo || b0 + 16 * NT - 1 > all_hi) {
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                bool seen[2] = {false, false};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const int j = e & 1, key = b0 + 16 * t + kk + (e >> 1) * 8;
                                    const bool ok = key <= qpos[j] && key >= wlo[j] && key < ke;
                                    sc[t][e] = ok ? sc[t][e] : -INFINITY;
                                    seen[e >> 1] |= ok;
                                }
                                // a key that neither of this lane's rows sees counts as zeros, whatever lies there
#pragma unroll
                                for (int h = 0; h < 2; ++h)
#pragma unroll
                                    for (int g = 0; g < NG; ++g) vs[t][h][g] = seen[h] ? vs[t][h][g] : 0u;
                            }
                        }
                        // The reference maximum moves only when some score of a row is more than 2^8 above it: until then no
                        // lane asks another
                        bool grown = false;
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int e = 0; e < 4; ++e) grown |= sc[t][e] > m_run[e & 1] + 8.f;
                        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                float mx = fmaxf(sc[0][j], sc[0][2 + j]);
                                if (NT == 2) mx = fmax3(mx, sc[NT - 1][j], sc[NT - 1][2 + j]);
                                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                                const bool g = mx > m_run[j] + 8.f;
                                const float f = g ? fast_exp2(m_run[j] - mx) : 1.f;
                                if (g) m_run[j] = mx;
                                l_run[j] *= f;
#pragma unroll
                                for (int i = 0; i < NG * TG; ++i) {
                                    o[i][j] *= f;
                                    o[i][2 + j] *= f;
                                }
#pragma unroll
                                for (int i = 0; i < NG; ++i) {
                                    psum[i][j] *= f;
                                    mid[i][j] *= f;
                                }
                            }
                        }
                        float muse[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) muse[j] = m_run[j] == -INFINITY ? 0.f : m_run[j];
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                sc[t][e] = fast_exp2(sc[t][e] - muse[e & 1]);
                                l_run[e & 1] += sc[t][e];
                            }
                        // O^T [16 dims x 8 rows] += V^T (P s)^T, a group at a time; A = V^T from the keys of rows 2 q4,
                        // 2 q4 + 1, 2 q4 + 8, 2 q4 + 9: a byte permute pairs two keys' numbers
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const uint8_t* va = stg + t * T::kTile + g4_key_of(2 * q4) * T::kPitch + F::kPart + g8 * (F::kGroup / 16);
                            const uint8_t* vb = stg + t * T::kTile + g4_key_of(2 * q4 + 1) * T::kPitch + F::kPart + g8 * (F::kGroup / 16);
#pragma unroll
                            for (int g = 0; g < NG; ++g) {
                                const int off = g * (F::kGroup / 2);
                                uint32_t wa, wb, wc, wd;
                                if constexpr (F::kGroup == 64) {
                                    wa = *reinterpret_cast<const uint32_t*>(va + off);
                                    wb = *reinterpret_cast<const uint32_t*>(vb + off);
                                    wc = *reinterpret_cast<const uint32_t*>(va + 8 * T::kPitch + off);
                                    wd = *reinterpret_cast<const uint32_t*>(vb + 8 * T::kPitch + off);
                                } else {
                                    wa = *reinterpret_cast<const uint16_t*>(va + off);
                                    wb = *reinterpret_cast<const uint16_t*>(vb + off);
                                    wc = *reinterpret_cast<const uint16_t*>(va + 8 * T::kPitch + off);
                                    wd = *reinterpret_cast<const uint16_t*>(vb + 8 * T::kPitch + off);
                                }
                                float ps[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float sv = bf16_lo(vs[t][e >> 1][g]);
                                    ps[e] = sc[t][e] * (sv * 0x1p64f);
                                    mid[g][e & 1] = fmaf(sc[t][e], fmaf(7.5f, sv, bf16_hi(vs[t][e >> 1][g])), mid[g][e & 1]);
                                }
                                const uint32_t pb0 = movmatrix_t(pack_bf16(ps[0], ps[1])), pb1 = movmatrix_t(pack_bf16(ps[2], ps[3]));
                                const uint32_t ones[4] = {0x00010001u, 0x00010001u, 0x00010001u, 0x00010001u};
                                mma_bf16(psum[g], ones, pb0, pb1);
#pragma unroll
                                for (int half = 0; half < TG / 2; ++half) {
                                    const uint32_t u = half ? __byte_perm(wa, wb, 0x7632) : __byte_perm(wa, wb, 0x5410);
                                    const uint32_t v = half ? __byte_perm(wc, wd, 0x7632) : __byte_perm(wc, wd, 0x5410);
                                    const uint32_t u8 = u >> 8, v8 = v >> 8;
                                    const uint32_t f0[4] = {u & 0x000f000fu, u & 0x00f000f0u, v & 0x000f000fu, v & 0x00f000f0u};
                                    const uint32_t f1[4] = {u8 & 0x000f000fu, u8 & 0x00f000f0u, v8 & 0x000f000fu, v8 & 0x00f000f0u};
                                    mma_bf16(o[g * TG + 2 * half], f0, pb0, pb1);
                                    mma_bf16(o[g * TG + 2 * half + 1], f1, pb0, pb1);
                                }
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[st]);
            }
            // ---- results of this warp's rows ----
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int x = 4; x < 32; x *= 2) {
                    l_run[j] += __shfl_xor_sync(0xffffffffu, l_run[j], x);
#pragma unroll
                    for (int g = 0; g < NG; ++g) mid[g][j] += __shfl_xor_sync(0xffffffffu, mid[g][j], x);
                }
            }
            if (!s_abort && head_ok) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (!rv[j]) continue;
                    const int R = rb + 2 * q4 + j;
                    const bool whole = w.num_splits == 1;
                    const float inv = !whole ? 1.f : l_run[j] > 0.f ? 1.f / l_run[j] : 0.f;
                    __nv_bfloat16* dst = a.out + ((size_t)(q_start + R / G) * a.num_q_heads + head * G + R % G) * D;
                    float* po = a.partial_o + ((size_t)self * kRowO + warp * kDecodeRows + 2 * q4 + j) * D;
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        // (both rows of psum's columns hold the sum)
                        const float base = fmaf(-7.5f * kUp, psum[g][j], mid[g][j]);
#pragma unroll
                        for (int t = 0; t < TG; ++t) {
                            const int d = g * F::kGroup + g8 * (F::kGroup / 8) + 2 * t;
                            const float x = fmaf(o[g * TG + t][j], kUp, base) * inv, y = fmaf(o[g * TG + t][2 + j], kUp * 0.0625f, base) * inv;
                            if (whole)
                                *reinterpret_cast<uint32_t*>(dst + d) = pack_bf16(x, y);
                            else
                                *reinterpret_cast<float2*>(po + d) = make_float2(x, y);
                        }
                    }
                    if (!whole && g8 == 0)
                        *reinterpret_cast<float2*>(a.partial_ml + ((size_t)self * kRowO + warp * kDecodeRows + 2 * q4 + j) * 2) =
                            make_float2(m_run[j], l_run[j]);
                }
            }
        }
        pipe += n_blocks;
        __syncthreads();
        if (s_abort) break;
        if (w.num_splits == 1) continue;
        // ---- the last CTA of the group joins its pieces ----
        __threadfence();
        __syncthreads();
        if (tid == 0) s_last = atomicAdd(&a.tickets[w.first_item], 1) == w.num_splits - 1;
        __syncthreads();
        if (!s_last) continue;
        __threadfence();
        if (!producer && warp < seg_heads) {
            const int head = h0 + warp;
            for (int R = w.row_begin; R < min(n_rows, w.row_begin + kDecodeRows); ++R) {
                const size_t row = (size_t)w.first_item * kRowO + warp * kDecodeRows + (R - w.row_begin);
                float M = -INFINITY, L = 0.f, acc[D / 32];
#pragma unroll
                for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
                for (int sp = 0; sp < w.num_splits; ++sp)
                    M = fmaxf(M, __ldcg(a.partial_ml + (row + (size_t)sp * kRowO) * 2));
                const float Mu = M == -INFINITY ? 0.f : M;
                for (int sp = 0; sp < w.num_splits; ++sp) {
                    const size_t at = row + (size_t)sp * kRowO;
                    const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.partial_ml) + at);
                    const float f = fast_exp2(ml.x - Mu);
                    L += f * ml.y;
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) acc[i] += f * __ldcg(a.partial_o + at * D + i * 32 + lane);
                }
                const float inv = L > 0.f ? 1.f / L : 0.f;
                __nv_bfloat16* dst = a.out + ((size_t)(q_start + R / G) * a.num_q_heads + head * G + R % G) * D;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) dst[i * 32 + lane] = __float2bfloat16_rn(acc[i] * inv);
            }
        }
        if (tid == 0) a.tickets[w.first_item] = 0;
    }
    // after an abort, wait (bounded) until no bulk copy can still land in this CTA's memory
    if (producer && lane == 0 && s_abort) {
        for (uint32_t i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i) mbar_wait(&full[i % STAGES], (i / STAGES) & 1, err);
    }
    if (tid == 0 && (int)blockIdx.x < n_static) atomicAdd(&hdr->next_item[0], 1);
    // started early beside the prefill grid: end after it, so that later launches see the plain order
    if (tid == 0) pdl_wait();
}

template <int D, int HG>
static cudaError_t launch_dec(const RpaArgs& a, int num_sms, cudaStream_t stream, int* per_sm_out) {
    using T = G4Dec<D, HG>;
    auto kern = g4_decode_kernel<D, HG>;
    static int per_sm[64] = {};  // (by device: the attribute is the device's)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (per_sm[dev] == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
        if (e != cudaSuccess) return e;
        int n = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, T::kThreads, T::kSmem);
        if (e != cudaSuccess) return e;
        per_sm[dev] = n > 0 ? n : 1;
    }
    if (per_sm_out) {
        *per_sm_out = per_sm[dev];
        return cudaSuccess;
    }
    CUtensorMap tkv;
    memset(&tkv, 0, sizeof tkv);
    const int ps = a.page_size;
    const long long tokens = (long long)a.total_num_pages * ps;
    const int boxes = (ps & (ps - 1)) == 0 && ps >= 16 && tokens <= INT32_MAX &&
                      make_tmap_heads(&tkv, a.kv_pages, G4<D>::kRow, a.num_kv_heads, (uint64_t)tokens, T::kPitch, 16, HG);
    ProfScope prof("rpa_g4_decode", stream);
    return launch_pdl(kern, dim3(num_sms * per_sm[dev]), dim3(T::kThreads), T::kSmem, stream, a.overlap != 0, a, tkv, boxes);
}

static cudaError_t dispatch(const RpaArgs& a, int num_sms, cudaStream_t stream, int* per_sm_out) {
    switch (a.head_dim) {
        case 64: return launch_dec<64, 4>(a, num_sms, stream, per_sm_out);
        case 128: return launch_dec<128, 4>(a, num_sms, stream, per_sm_out);
        // Two heads a CTA leave four warps an SM that compute (64 decodes that see 1024 to 4096 keys of 8 heads, with a
        // soft cap: 180 us; four heads a CTA 128, although 118 bytes of their 168 registers a thread spill), but half of four would
        // idle where a cache has two heads.
        case 256: return a.decode_heads == 4 ? launch_dec<256, 4>(a, num_sms, stream, per_sm_out) : launch_dec<256, 2>(a, num_sms, stream, per_sm_out);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_g4_decode(const RpaArgs& a, int num_sms, cudaStream_t stream) { return dispatch(a, num_sms, stream, nullptr); }

int g4_decode_ctas_per_sm(const RpaArgs& a) {
    int n = 0;
    return dispatch(a, 0, nullptr, &n) == cudaSuccess ? n : 0;
}

}  // namespace rpa
