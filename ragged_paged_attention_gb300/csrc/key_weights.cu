// What each cached key gets of a batch's attention (rpa_key_weights), for sm_103a:
//
//   w_out[key] = keep w_in[key] + sum over the sequence's queries and the group's q heads of 2^(c s - L),
//   L = log2 of the row's sum of 2^(c s) over the keys it sees, c = sm_scale log2(e), s = q.k (its soft cap, too).
//
// Behind a plan one kernel finds each row's maximum and sum over pieces of its keys. Sequences of up to 16 rows a KV head (decodes)
// leave their scores there, 16 bytes a key for 4 rows beside K's 256 (bf16, D = 128), and a light kernel adds them up;
// for the others a third computes the scores again, knowing L. Items are a warp's: 16 keys fill the M side of m16n8k16, 16
// query rows (G heads x tokens) two N sides; a warp copies its K rows (no V) by cp.async a few stages ahead and
// waits for nobody else. A row's running maximum and sum stay in each lane on the keys it holds, and meet once an item.
// Scores are exact products in float32: bf16 operands, or the 4-bit numbers as bf16 subnormals with their groups'
// accumulators apart (g4_decode.cu). Maxima, sums and L are float32; exponentials are ex2.approx (2^-22), soft caps tanhf.
//
// 96 decodes over 2000 to 8192 keys, 32/8 heads of 128, bf16: 192 us for the statistics (1 GB of K in rows of 256 bytes, every
// other 256 of a page: 5.3 TB/s) and 47 us for the sums (16 bytes of scores and 8 of weights a key; bound by the latency
// of page table, scores and weights in a row). With the scores computed again instead of stored the call took 561 us,
// not 241.
#include "common.cuh"
#include "g4.cuh"
#include "kernels.h"
#include "profile.h"

namespace rpa {

constexpr int kKwWarps = 4;              // of a block
constexpr int kKwStages = 4;
constexpr int kKwBK = 16;                // keys a stage

template <int D, bool IS_G4>
struct Kw {
    // a key's bytes of one head in a stage, and the pitch: rows of 16 more bytes for ldmatrix; 4-bit rows (K's numbers, then
    // the 16 bytes that start with K's scales) so that the loads of eight rows touch every bank once
    static constexpr int kBytes = IS_G4 ? D / 2 + 16 : 2 * D;
    static constexpr int kPitch = IS_G4 ? (D == 64 ? 48 : D == 128 ? 96 : 160) : 2 * D + 16;
    static constexpr int kUnits = kBytes / 16;
    static constexpr int kStage = kKwBK * kPitch;
    static constexpr int kSmem = kKwWarps * kKwStages * kStage;
};

// One warp's reader of 16-key stages of one head, and their scores against up to 16 query rows.
template <int D, bool IS_G4>
struct KwScores {
    using T = Kw<D, IS_G4>;
    using F = G4<D>;
    static constexpr int NG = F::NG, KW = F::kGroup / 32;
    uint32_t qb[2][D / 16][2];             // Q^T as B fragments, two tiles of 8 rows
    float qsum[2][IS_G4 ? NG : 1][2];      // 4-bit caches: sums of the row over a group, and
    float colmul[2][2];                    // the power of two that brings its scores back

    // Rows row0 .. row0 + 15 of the sequence's (row = token * G + head of the group); rows that are not there are zeros.
    __device__ __forceinline__ void load_q(const KwArgs& a, int q_start, int head, int G, int row0, int n_rows) {
        const int lane = threadIdx.x & 31, g8 = lane >> 2, q4 = lane & 3;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            const int R = row0 + 8 * nt + g8;
            const bool rv = R < n_rows;
            const __nv_bfloat16* row = a.q + ((size_t)(q_start + (rv ? R / G : 0)) * a.num_q_heads + head * G + (rv ? R % G : 0)) * D;
            if constexpr (!IS_G4) {
                const uint32_t* w = reinterpret_cast<const uint32_t*>(row);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    qb[nt][ks][0] = rv ? __ldg(w + ks * 8 + q4) : 0u;
                    qb[nt][ks][1] = rv ? __ldg(w + ks * 8 + 4 + q4) : 0u;
                }
            } else {
                // (g4_decode.cu: a lane's 8 dims of a word, the odd ones of either pair a 16th)
                const uint4* w = reinterpret_cast<const uint4*>(row);
                uint4 raw[NG * KW];
                float mabs = 0.f;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    float sum = 0.f;
#pragma unroll
                    for (int wd = 0; wd < KW; ++wd) {
                        const uint4 v = rv ? __ldg(w + (g * F::kGroup + q4 * (F::kGroup / 4)) / 8 + wd) : make_uint4(0, 0, 0, 0);
                        raw[g * KW + wd] = v;
                        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            sum += bf16_lo(x[e]) + bf16_hi(x[e]);
                            mabs = fmax3(mabs, fabsf(bf16_lo(x[e])), fabsf(bf16_hi(x[e])));
                        }
                    }
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
                    for (int j = 0; j < 2; ++j) qsum[nt][g][j] = __shfl_sync(0xffffffffu, sum, (2 * q4 + j) * 4);
                }
                mabs = fmaxf(mabs, __shfl_xor_sync(0xffffffffu, mabs, 1));
                mabs = fmaxf(mabs, __shfl_xor_sync(0xffffffffu, mabs, 2));
                int ex = 0;
                frexpf(mabs, &ex);
                const int k = max(6, min(120, 120 - ex));
                const float qs = ldexpf(1.f, k), rowmul = ldexpf(1.f, 133 - k);
                auto scaled = [&](uint32_t lo, uint32_t hi, float f) {
                    return pack_bf16(fminf(fmaxf(__uint_as_float(lo) * f, -0x1p126f), 0x1p126f),
                                     fminf(fmaxf(__uint_as_float(hi) * f, -0x1p126f), 0x1p126f));
                };
#pragma unroll
                for (int i = 0; i < NG * KW; ++i) {
                    const uint4 v = raw[i];
                    qb[nt][2 * i][0] = scaled(v.x << 16, v.z << 16, qs);
                    qb[nt][2 * i][1] = scaled(v.x & 0xffff0000u, v.z & 0xffff0000u, qs * 0.0625f);
                    qb[nt][2 * i + 1][0] = scaled(v.y << 16, v.w << 16, qs);
                    qb[nt][2 * i + 1][1] = scaled(v.y & 0xffff0000u, v.w & 0xffff0000u, qs * 0.0625f);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) colmul[nt][j] = __shfl_sync(0xffffffffu, rowmul, (2 * q4 + j) * 4);
            }
        }
    }

    // Sixteen keys from `key` on (those below ke) of one head, on their way into a stage. `page_lane`: lane i's page
    // of key + i.
    __device__ __forceinline__ static void ask(const KwArgs& a, uint8_t* stage, int head, int key, int ke, int page_lane) {
        const int lane = threadIdx.x & 31;
        const uint8_t* kv = static_cast<const uint8_t*>(a.kv_pages);
        constexpr size_t kHead = IS_G4 ? F::kRow : 4 * D;  // bytes of a key's K and V of one head
        // lane i's row, passed on to the lanes that copy it
        const int k = key + lane;
        const size_t slot = (size_t)page_lane * a.page_size + k % a.page_size;
        const unsigned long long row = reinterpret_cast<unsigned long long>(kv + (slot * a.num_kv_heads + head) * kHead);
        constexpr int kAll = kKwBK * T::kUnits;
#pragma unroll
        for (int i0 = 0; i0 < kAll; i0 += 32) {
            const int i = i0 + lane, r = i / T::kUnits, c = i % T::kUnits;
            const unsigned long long src = __shfl_sync(0xffffffffu, row, r & 15);
            if (i < kAll && key + r < ke) {
                const int off = IS_G4 && c == T::kUnits - 1 ? F::kParams : c * 16;
                cp_async16(smem_u32(stage + r * T::kPitch + c * 16), reinterpret_cast<const uint8_t*>(src) + off, true);
            }
        }
    }

    // The scores of a stage: sc[nt][e] of key g8 + 8 (e >> 1) and row 8 nt + 2 q4 + (e & 1).
    __device__ __forceinline__ void scores(const uint8_t* stage, bool two, float (&sc)[2][4]) const {
        const int lane = threadIdx.x & 31, g8 = lane >> 2, q4 = lane & 3;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
        if constexpr (!IS_G4) {
            const uint32_t ka = smem_u32(stage) + ((lane & 7) + ((lane >> 3) & 1) * 8) * T::kPitch + (lane >> 4) * 16;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t f[4];
                ldsm_x4(ka + ks * 32, f[0], f[1], f[2], f[3]);
                mma_bf16(sc[0], f, qb[0][ks][0], qb[0][ks][1]);
                if (two) mma_bf16(sc[1], f, qb[1][ks][0], qb[1][ks][1]);
            }
        } else {
            const uint8_t* r0 = stage + g8 * T::kPitch;
            const uint8_t* r1 = r0 + 8 * T::kPitch;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const int off = g * (F::kGroup / 2) + q4 * (F::kGroup / 8);
                float acc[2][4] = {};
#pragma unroll
                for (int wd = 0; wd < KW; ++wd) {
                    const uint32_t u = *reinterpret_cast<const uint32_t*>(r0 + off + 4 * wd), v = *reinterpret_cast<const uint32_t*>(r1 + off + 4 * wd);
                    const uint32_t u8 = u >> 8, v8 = v >> 8;
                    const uint32_t f0[4] = {u & 0x000f000fu, v & 0x000f000fu, u & 0x00f000f0u, v & 0x00f000f0u};
                    const uint32_t f1[4] = {u8 & 0x000f000fu, v8 & 0x000f000fu, u8 & 0x00f000f0u, v8 & 0x00f000f0u};
                    const int i = 2 * (g * KW + wd);
                    mma_bf16(acc[0], f0, qb[0][i][0], qb[0][i][1]);
                    mma_bf16(acc[0], f1, qb[0][i + 1][0], qb[0][i + 1][1]);
                    if (two) {
                        mma_bf16(acc[1], f0, qb[1][i][0], qb[1][i][1]);
                        mma_bf16(acc[1], f1, qb[1][i + 1][0], qb[1][i + 1][1]);
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t sm = *reinterpret_cast<const uint32_t*>((h ? r1 : r0) + D / 2 + 4 * g);
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            sc[nt][2 * h + j] = fmaf(bf16_lo(sm), acc[nt][2 * h + j] * colmul[nt][j], fmaf(bf16_hi(sm), qsum[nt][g][j], sc[nt][2 * h + j]));
                }
            }
        }
    }
};

// A score in log2 units.
__device__ __forceinline__ float kw_log2(const KwArgs& a, float s) {
    s *= a.sm_scale;
    if (a.soft_cap != 0.f) s = a.soft_cap * tanhf(s / a.soft_cap);
    return s * kLog2e;
}

struct KwSeq {
    int q_start, q_len, kv_len, n_rows, tiles;
};
__device__ __forceinline__ KwSeq kw_seq(const KwArgs& a, int s, int G) {
    KwSeq q;
    q.q_start = a.cu_q_lens[s];
    q.q_len = a.cu_q_lens[s + 1] - q.q_start;
    q.kv_len = a.kv_lens[s];
    q.n_rows = q.q_len * G;
    q.tiles = cdiv(q.n_rows, 16);
    return q;
}
// Keys that rows row0 .. row0 + 15 see between them: [lo, hi).
__device__ __forceinline__ void kw_range(const KwArgs& a, const KwSeq& q, int G, int row0, int& lo, int& hi) {
    const int last = min(q.n_rows, row0 + 16) - 1, p0 = q.kv_len - q.q_len + row0 / G;
    hi = q.kv_len - q.q_len + last / G + 1;
    lo = a.sliding_window > 0 ? max(0, p0 - a.sliding_window + 1) : 0;
}

// Rows a key of stored scores.
__device__ __forceinline__ int kw_row_slots(int n_rows) { return n_rows <= 4 ? 4 : n_rows <= 8 ? 8 : 16; }

// Ends of the kernels' items, a sequence after another, the keys of a piece, and where sequences of one row tile leave
// their scores.  A chain of latencies: few threads, whose barriers are short (1024 of them: 16 us), the lengths in the same
// round trip as their count, and two numbers a scan.
constexpr int kKwPlan = 256;
__global__ void __launch_bounds__(kKwPlan) kw_plan_kernel(const __grid_constant__ KwArgs a) {
    __shared__ long long scan[40];
    __shared__ float red[4][8];
    const int tid = threadIdx.x, lane = tid & 31, G = a.num_q_heads / a.num_kv_heads;
    pdl_launch_dependents();  // (the next kernel waits for this one's end)
    pdl_wait();               // (the stream's earlier work may be writing the lengths)
    const int mine = min(tid, a.max_num_seqs - 1);
    int c0 = a.cu_q_lens[mine], c1 = a.cu_q_lens[mine + 1], k = a.kv_lens[mine];
    int num = a.num_seqs[0];
    if (num < 0 || num > a.max_num_seqs) {
        if (tid == 0) set_error(&a.hdr->error_bits, RPA_DEV_ERR_NUM_SEQS);
        num = 0;
    }
    auto shape = [&](int s, int& ql, int& kl) {
        ql = kl = 0;
        if (s >= num) return;
        if (s != tid) {
            c0 = a.cu_q_lens[s];
            c1 = a.cu_q_lens[s + 1];
            k = a.kv_lens[s];
        }
        uint32_t bad = 0;
        if (c0 < 0 || c1 < c0 || c1 > a.max_num_tokens)
            bad = RPA_DEV_ERR_TOKENS;
        else if (c1 - c0 > k)
            bad = RPA_DEV_ERR_Q_LEN;
        else if (k > 0 && (k - 1) / a.page_size >= a.pages_per_seq)
            bad = RPA_DEV_ERR_KV_LEN;
        if (bad) {
            set_error(&a.hdr->error_bits, bad);
            return;
        }
        ql = c1 - c0;
        kl = ql ? k : 0;
    };
    // the batch's work, cut into about as many pieces as keep the warps (and, for the tensor cores' kernels, the CTAs)
    // busy: keys x tiles of 16 rows; keys of sequences of one tile; blocks x tiles of 128; blocks
    float work[4] = {0.f, 0.f, 0.f, 0.f};
    auto count = [&](int ql, int kl) {
        if (a.use_tc && ql * G > 16) {
            work[2] += (float)cdiv(ql * G, 128) * (float)cdiv(kl, 128);
            work[3] += (float)cdiv(kl, 128);
        } else {
            work[0] += (float)cdiv(ql * G, 16) * (float)kl;
            if (ql * G <= 16) work[1] += (float)kl;
        }
    };
    int ql0, kl0;
    shape(tid, ql0, kl0);
    count(ql0, kl0);
    for (int s = tid + kKwPlan; s < num; s += kKwPlan) {
        int ql, kl;
        shape(s, ql, kl);
        count(ql, kl);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        work[i] = warp_sum(work[i]);
        if (lane == 0) red[i][tid >> 5] = work[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v = 0.f;
#pragma unroll
        for (int j = 0; j < kKwPlan / 32; ++j) v += red[i][j];
        work[i] = v * (float)a.num_kv_heads;
    }
    const int piece = max(kKwMinPiece, (int)min((double)work[0] / kKwTarget, 1e9) / kKwBK * kKwBK + kKwBK);
    const int longest = min(kKwLong, max(64, ((int)min((double)work[1] / kKwTarget, 1e9) / 32 + 1) * 32));
    const int tc_piece = 1 + (int)min((double)work[2] / kKwTcTarget, 1e9);
    const int tc_chunk = max(1, min(kKwTcChunk, (int)(work[3] / (kKwTcTarget / 2))));
    int base_a = 0, base_b = 0, base_c = 0, base_d = 0, base_e = 0;
    long long base_s = 0;  // scores, in units of 64
    for (int s0 = 0; s0 < num; s0 += kKwPlan) {
        int ql = ql0, kl = kl0;
        if (s0) shape(s0 + tid, ql, kl);
        const int rows = ql * G;
        const bool tc = a.use_tc && rows > 16;
        // (scores: 32 bits are enough for what fits the workspace; a sequence with more has none)
        const long long units = rows > 0 && rows <= 16 ? (long long)cdiv(kl, 16) * kw_row_slots(rows) / 4 * a.num_kv_heads : 0;
        const long long want = units * 64 <= a.max_scores ? units : 0;
        long long total;
        const int na = tc ? 0 : cdiv(rows, 16) * a.num_kv_heads * cdiv(kl, piece);
        const long long sa = block_exclusive_scan((want << 32) | na, scan, &total);
        const long long at = base_s + (sa >> 32);
        const bool stored = want > 0 && (at + want) * 64 <= a.max_scores;
        base_s += total >> 32;
        const int total_a = (int)(total & 0xffffffffll);
        const int nb = ql && !stored && !tc ? a.num_kv_heads * cdiv(kl, kKwChunk) : 0, nc = stored ? a.num_kv_heads * cdiv(kl, longest) : 0;
        const long long bc = block_exclusive_scan(((long long)nb << 32) | nc, scan, &total);
        const int total_b = (int)(total >> 32), total_c = (int)(total & 0xffffffffll);
        long long total_de = 0, de = 0;
        const int blocks = cdiv(kl, 128), nd = tc ? cdiv(rows, 128) * a.num_kv_heads * cdiv(blocks, tc_piece) : 0;
        const int ne = tc ? a.num_kv_heads * cdiv(blocks, tc_chunk) : 0;
        if (work[3] > 0.f) de = block_exclusive_scan(((long long)nd << 32) | ne, scan, &total_de);
        if (s0 + tid < num) {
            a.ends_a[s0 + tid] = base_a + (int)(sa & 0xffffffffll) + na;
            a.ends_b[s0 + tid] = base_b + (int)(bc >> 32) + nb;
            a.ends_c[s0 + tid] = base_c + (int)(bc & 0xffffffffll) + nc;
            a.score_at[s0 + tid] = stored ? (int)at : -1;
            a.ends_d[s0 + tid] = base_d + (int)(de >> 32) + nd;
            a.ends_e[s0 + tid] = base_e + (int)(de & 0xffffffffll) + ne;
        }
        base_a += total_a;
        base_b += total_b;
        base_c += total_c;
        base_d += (int)(total_de >> 32);
        base_e += (int)(total_de & 0xffffffffll);
    }
    if (tid == 0) {
        if (base_a > a.max_items || base_d > a.max_tc_items) {  // (only sequences that claim the same tokens make so many)
            set_error(&a.hdr->error_bits, RPA_DEV_ERR_TOKENS);
            base_a = base_b = base_c = base_d = base_e = 0;
        }
        a.tc[0] = base_d;
        a.tc[1] = base_e;
        a.tc[2] = tc_piece;
        a.tc[3] = tc_chunk;
        a.tc[4] = a.tc[5] = 0;
        a.tc[6] = longest;
        a.hdr->num_items[0] = base_a;
        a.hdr->num_items[1] = base_b;
        a.hdr->num_items[2] = num;
        a.hdr->num_items[3] = base_c;
        a.hdr->chunk_keys = piece;
        a.hdr->next_item[0] = a.hdr->next_item[1] = a.hdr->next_item[2] = 0;
    }
}

__device__ __forceinline__ int kw_take(int* counter) {
    int i = 0;
    if ((threadIdx.x & 31) == 0) i = atomicAdd(counter, 1);
    return __shfl_sync(0xffffffffu, i, 0);
}

// Lane i's page of key + i (0 where there is none to read; a bad one is recorded and replaced).
__device__ __forceinline__ int kw_page(const KwArgs& a, const int* tbl, int key, int ke) {
    const int k = key + (threadIdx.x & 31);
    int page = 0;
    if ((threadIdx.x & 31) < kKwBK && k < ke) {
        page = __ldg(tbl + k / a.page_size);
        if ((unsigned)page >= (unsigned)a.total_num_pages) {
            set_error(&a.hdr->error_bits, RPA_DEV_ERR_PAGE);
            page = 0;
        }
    }
    return page;
}

// Walks the stages of keys [k0, ke): copies kKwStages - 1 ahead, body(first key, stage) on each.
template <int D, bool IS_G4, typename Body>
__device__ __forceinline__ void kw_walk(const KwArgs& a, uint8_t* ring, const int* tbl, int head, int k0, int ke, Body&& body) {
    using T = Kw<D, IS_G4>;
    const int n = cdiv(ke - k0, kKwBK);
    auto ask = [&](int j, int page) {
        if (j < n) KwScores<D, IS_G4>::ask(a, ring + (j % kKwStages) * T::kStage, head, k0 + j * kKwBK, ke, page);
        cp_async_commit();
    };
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kKwStages - 1; ++j) ask(j, kw_page(a, tbl, k0 + j * kKwBK, ke));
    int page = kw_page(a, tbl, k0 + (kKwStages - 1) * kKwBK, ke);
    for (int j = 0; j < n; ++j) {
        cp_async_wait<kKwStages - 2>();
        __syncwarp();
        ask(j + kKwStages - 1, page);
        page = kw_page(a, tbl, k0 + (j + kKwStages) * kKwBK, ke);
        body(j, ring + (j % kKwStages) * T::kStage);
    }
    cp_async_wait<0>();
}

// Rows' maxima (log2 units) and sums over a piece of their keys.
template <int D, bool IS_G4>
__global__ void __launch_bounds__(kKwWarps * 32) kw_stats_kernel(const __grid_constant__ KwArgs a) {
    using T = Kw<D, IS_G4>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g8 = lane >> 2, q4 = lane & 3, G = a.num_q_heads / a.num_kv_heads;
    uint8_t* ring = smem + warp * kKwStages * T::kStage;
    // rows that are never copied stay finite
    for (int i = threadIdx.x * 16; i < T::kSmem; i += blockDim.x * 16) *reinterpret_cast<uint4*>(smem + i) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    pdl_launch_dependents();  // (the kernels behind wait for this grid's end)
    pdl_wait();
    const int n_items = a.hdr->num_items[0], num = a.hdr->num_items[2], piece = a.hdr->chunk_keys;
    while (true) {
        const int item = kw_take(&a.hdr->next_item[0]);
        if (item >= n_items) break;
        int first;
        const int s = kw_find(a.ends_a, num, item, first);
        const KwSeq q = kw_seq(a, s, G);
        const int splits = cdiv(q.kv_len, piece), rel = item - first;
        const int split = rel % splits, tile = rel / splits % q.tiles, head = rel / (splits * q.tiles), row0 = 16 * tile;
        int lo, hi;
        kw_range(a, q, G, row0, lo, hi);
        const int store = a.score_at[s], slots = kw_row_slots(q.n_rows);
        // (stored scores are there for every key, also those that a window hides)
        const int k0 = max(split * piece, store >= 0 ? 0 : lo / kKwBK * kKwBK), ke = min(hi, (split + 1) * piece);
        const bool two = q.n_rows - row0 > 8;
        float* to = store >= 0 ? a.scores + (size_t)store * 64 + (size_t)head * cdiv(q.kv_len, 16) * 16 * slots + 2 * q4 : nullptr;
        float m[2][2], l[2][2];
        int at[2][2];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                m[nt][j] = -INFINITY;
                l[nt][j] = 0.f;
                const int R = row0 + 8 * nt + 2 * q4 + j;
                at[nt][j] = R < q.n_rows ? q.kv_len - q.q_len + R / G : -1;  // the row's position
            }
        if (k0 < ke) {
            KwScores<D, IS_G4> x;
            x.load_q(a, q.q_start, head, G, row0, q.n_rows);
            kw_walk<D, IS_G4>(a, ring, a.page_indices + (size_t)s * a.pages_per_seq, head, k0, ke, [&](int j, const uint8_t* stage) {
                float sc[2][4];
                x.scores(stage, two, sc);
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    if (nt == 1 && !two) break;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = k0 + j * kKwBK + g8 + 8 * (e >> 1), p = at[nt][e & 1];
                        const bool seen = key <= p && key < ke && (a.sliding_window == 0 || key > p - a.sliding_window);
                        sc[nt][e] = seen ? kw_log2(a, sc[nt][e]) : -INFINITY;
                    }
                    if (to && 8 * nt + 2 * q4 < slots) {
                        float* at_key = to + (size_t)(k0 + j * kKwBK + g8) * slots + 8 * nt;
                        *reinterpret_cast<float2*>(at_key) = make_float2(sc[nt][0], sc[nt][1]);
                        *reinterpret_cast<float2*>(at_key + 8 * slots) = make_float2(sc[nt][2], sc[nt][3]);
                    }
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float mx = fmaxf(sc[nt][c], sc[nt][2 + c]);
                        if (mx > m[nt][c]) {
                            l[nt][c] *= fast_exp2(m[nt][c] - mx);
                            m[nt][c] = mx;
                        }
                        const float u = m[nt][c] == -INFINITY ? 0.f : m[nt][c];
                        l[nt][c] += fast_exp2(sc[nt][c] - u) + fast_exp2(sc[nt][2 + c] - u);
                    }
                }
            });
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float M = m[nt][j];
#pragma unroll
                for (int o = 4; o < 32; o *= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
                float v = M == -INFINITY ? 0.f : l[nt][j] * fast_exp2(m[nt][j] - M);
#pragma unroll
                for (int o = 4; o < 32; o *= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (g8 == 0) a.stats[(size_t)item * 16 + 8 * nt + 2 * q4 + j] = make_float2(M, v);
            }
    }
}

// L of row lane of a tile (lanes below 16), from its pieces; infinity for a row that is not there.
__device__ __forceinline__ float kw_norm(const KwArgs& a, int first_a, int head, int tile, const KwSeq& q, int splits) {
    const int lane = threadIdx.x & 31;
    if (lane >= 16 || 16 * tile + lane >= q.n_rows) return INFINITY;
    const float2* st = a.stats + ((size_t)first_a + ((size_t)head * q.tiles + tile) * splits) * 16 + lane;
    float M = -INFINITY, sum = 0.f;
#pragma unroll 8
    for (int i = 0; i < splits; ++i) {
        const float2 v = st[(size_t)i * 16];
        const float n = fmaxf(M, v.x), u = n == -INFINITY ? 0.f : n;
        sum = sum * fast_exp2(M - u) + v.y * fast_exp2(v.x - u);
        M = n;
    }
    return M + log2f(sum);
}

// The keys of sequences whose scores are stored: a warp takes up to kKwLong keys of a head, a key a lane.
template <int R>
__device__ __forceinline__ void kw_finish(const KwArgs& a, float L, const float* scores, const int* tbl, int head, int c0, int c1) {
    const int lane = threadIdx.x & 31;
    float Lr[R];
#pragma unroll
    for (int r = 0; r < R; ++r) Lr[r] = __shfl_sync(0xffffffffu, L, r);
#pragma unroll 4
    for (int key = c0 + lane; key < c1; key += 32) {
        const float4* p = reinterpret_cast<const float4*>(scores + (size_t)key * R);
        float v = 0.f;
#pragma unroll
        for (int r = 0; r < R / 4; ++r) {
            const float4 x = __ldcs(p + r);
            v += (fast_exp2(x.x - Lr[4 * r]) + fast_exp2(x.y - Lr[4 * r + 1])) + (fast_exp2(x.z - Lr[4 * r + 2]) + fast_exp2(x.w - Lr[4 * r + 3]));
        }
        const int p_at = key / a.page_size, page = __ldg(tbl + p_at);
        if ((unsigned)page < (unsigned)a.total_num_pages) {
            const size_t o = ((size_t)page * a.num_kv_heads + head) * a.page_size + (key - p_at * a.page_size);
            a.weights_out[o] = a.keep == 0.f ? v : fmaf(a.keep, a.weights[o], v);
        }
    }
}
__global__ void __launch_bounds__(kKwWarps * 32) kw_finish_kernel(const __grid_constant__ KwArgs a) {
    const int G = a.num_q_heads / a.num_kv_heads;
    pdl_launch_dependents();  // (the kernel behind works on other sequences' keys, and waits for this one's end)
    pdl_wait();
    const int n_items = a.hdr->num_items[3], num = a.hdr->num_items[2], piece = a.hdr->chunk_keys, longest = a.tc[6];
    while (true) {
        const int item = kw_take(&a.hdr->next_item[2]);
        if (item >= n_items) break;
        int first;
        const int s = kw_find(a.ends_c, num, item, first), first_a = s > 0 ? a.ends_a[s - 1] : 0, store = a.score_at[s];
        const KwSeq q = kw_seq(a, s, G);
        const int chunks = cdiv(q.kv_len, longest), rel = item - first, head = rel / chunks, c0 = rel % chunks * longest;
        const int c1 = min(q.kv_len, c0 + longest), slots = kw_row_slots(q.n_rows);
        const float L = kw_norm(a, first_a, head, 0, q, cdiv(q.kv_len, piece));
        const float* scores = a.scores + (size_t)store * 64 + (size_t)head * cdiv(q.kv_len, 16) * 16 * slots;
        const int* tbl = a.page_indices + (size_t)s * a.pages_per_seq;
        if (slots == 4)
            kw_finish<4>(a, L, scores, tbl, head, c0, c1);
        else if (slots == 8)
            kw_finish<8>(a, L, scores, tbl, head, c0, c1);
        else
            kw_finish<16>(a, L, scores, tbl, head, c0, c1);
    }
}

// Chunks of kKwChunk keys of a head: their weights over all of the sequence's rows.
template <int D, bool IS_G4>
__global__ void __launch_bounds__(kKwWarps * 32) kw_sum_kernel(const __grid_constant__ KwArgs a) {
    using T = Kw<D, IS_G4>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g8 = lane >> 2, q4 = lane & 3, G = a.num_q_heads / a.num_kv_heads;
    uint8_t* ring = smem + warp * kKwStages * T::kStage;
    for (int i = threadIdx.x * 16; i < T::kSmem; i += blockDim.x * 16) *reinterpret_cast<uint4*>(smem + i) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    pdl_wait();
    const int n_items = a.hdr->num_items[1], num = a.hdr->num_items[2], piece = a.hdr->chunk_keys;
    while (true) {
        const int item = kw_take(&a.hdr->next_item[1]);
        if (item >= n_items) break;
        int first, first_a;
        const int s = kw_find(a.ends_b, num, item, first);
        first_a = s > 0 ? a.ends_a[s - 1] : 0;
        const KwSeq q = kw_seq(a, s, G);
        const int chunks = cdiv(q.kv_len, kKwChunk), rel = item - first, head = rel / chunks, c0 = rel % chunks * kKwChunk;
        const int c1 = min(q.kv_len, c0 + kKwChunk), splits = cdiv(q.kv_len, piece);
        const int* tbl = a.page_indices + (size_t)s * a.pages_per_seq;
        float w[kKwChunk / kKwBK][2];
#pragma unroll
        for (int i = 0; i < kKwChunk / kKwBK; ++i) w[i][0] = w[i][1] = 0.f;
        for (int tile = 0; tile < q.tiles; ++tile) {
            const int row0 = 16 * tile;
            int lo, hi;
            kw_range(a, q, G, row0, lo, hi);
            if (hi <= c0 || lo >= c1) continue;
            const bool two = q.n_rows - row0 > 8;
            const float L = kw_norm(a, first_a, head, tile, q, splits);
            float Lc[2][2];
            int at[2][2];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = 8 * nt + 2 * q4 + j;
                    Lc[nt][j] = __shfl_sync(0xffffffffu, L, r);
                    at[nt][j] = row0 + r < q.n_rows ? q.kv_len - q.q_len + (row0 + r) / G : -1;
                }
            KwScores<D, IS_G4> x;
            x.load_q(a, q.q_start, head, G, row0, q.n_rows);
            kw_walk<D, IS_G4>(a, ring, tbl, head, c0, min(c1, hi), [&](int j, const uint8_t* stage) {
                float sc[2][4];
                x.scores(stage, two, sc);
                float add[2] = {0.f, 0.f};
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    if (nt == 1 && !two) break;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = c0 + j * kKwBK + g8 + 8 * (e >> 1), p = at[nt][e & 1];
                        const bool seen = key <= p && (a.sliding_window == 0 || key > p - a.sliding_window);
                        if (seen) add[e >> 1] += fast_exp2(kw_log2(a, sc[nt][e]) - Lc[nt][e & 1]);
                    }
                }
#pragma unroll
                for (int i = 0; i < kKwChunk / kKwBK; ++i)
                    if (i == j) {
                        w[i][0] += add[0];
                        w[i][1] += add[1];
                    }
            });
        }
        // a key's sum over the rows of its four lanes
#pragma unroll
        for (int i = 0; i < kKwChunk / kKwBK; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v = w[i][h];
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
                const int key = c0 + i * kKwBK + 8 * h + g8;
                if (q4 == 0 && key < c1) {
                    const int page = tbl[key / a.page_size];
                    if ((unsigned)page < (unsigned)a.total_num_pages) {
                        const size_t o = ((size_t)page * a.num_kv_heads + head) * a.page_size + key % a.page_size;
                        a.weights_out[o] = a.keep == 0.f ? v : fmaf(a.keep, a.weights[o], v);
                    }
                }
            }
    }
}

template <int D, bool IS_G4>
static cudaError_t launch_kw(const KwArgs& a, int num_sms, cudaStream_t stream) {
    using T = Kw<D, IS_G4>;
    static int per_sm[64][2] = {};  // (by device: the attribute is the device's)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    void (*kern[2])(const KwArgs) = {kw_stats_kernel<D, IS_G4>, kw_sum_kernel<D, IS_G4>};
    for (int i = 0; i < 2; ++i) {
        if (per_sm[dev][i]) continue;
        e = cudaFuncSetAttribute(kern[i], cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
        int n = 0;
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern[i], kKwWarps * 32, T::kSmem);
        if (e != cudaSuccess) return e;
        per_sm[dev][i] = n > 0 ? n : 1;
    }
    const bool pdl = !prof_enabled();
    {
        ProfScope ps("rpa_kw_stats", stream);
        e = launch_pdl(kern[0], dim3(num_sms * per_sm[dev][0]), dim3(kKwWarps * 32), T::kSmem, stream, pdl, a);
    }
    if (e != cudaSuccess) return e;
    {
        ProfScope ps("rpa_kw_finish", stream);
        e = launch_pdl(kw_finish_kernel, dim3(num_sms * 16), dim3(kKwWarps * 32), 0, stream, pdl, a);
    }
    // (so few query rows that every sequence has one tile, and the workspace room for all their scores: nothing is left)
    if (e != cudaSuccess || a.all_stored) return e;
    if (a.use_tc) {
        e = launch_kw_tc(a, D, false, num_sms, stream);
        if (e == cudaSuccess) e = launch_kw_tc(a, D, true, num_sms, stream);
        if (e != cudaSuccess || a.scores_fit) return e;
    }
    ProfScope ps("rpa_kw_sum", stream);
    return launch_pdl(kern[1], dim3(num_sms * per_sm[dev][1]), dim3(kKwWarps * 32), T::kSmem, stream, pdl, a);
}

cudaError_t launch_key_weights(const KwArgs& a, int head_dim, bool g4, int num_sms, cudaStream_t stream) {
    {
        ProfScope ps("rpa_kw_plan", stream);
        const cudaError_t e = launch_pdl(kw_plan_kernel, dim3(1), dim3(kKwPlan), 0, stream, !prof_enabled(), a);
        if (e != cudaSuccess) return e;
    }
    switch (head_dim) {
        case 64: return g4 ? launch_kw<64, true>(a, num_sms, stream) : launch_kw<64, false>(a, num_sms, stream);
        case 128: return g4 ? launch_kw<128, true>(a, num_sms, stream) : launch_kw<128, false>(a, num_sms, stream);
        case 256: return g4 ? launch_kw<256, true>(a, num_sms, stream) : launch_kw<256, false>(a, num_sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace rpa
