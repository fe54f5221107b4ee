// Rotary positions (rope_apply) and the cache write that turns its keys (rpa_rope_update_kv_cache),
// for sm_103a.
//
// Both only move memory: a turned element costs two fused multiply-adds against four bytes.
// rope_apply of 8191 tokens, 32 + 8 heads of 128: 28.7 us in a graph, 0.87 of the copy rate; the cache write of
// 4 x 4096 tokens, 32 + 8 + 8 heads of 128: bf16 70, fp8 62, int8 64, int4 65 us.
#include "common.cuh"
#include "kernels.h"
#include "profile.h"
#include "rope.cuh"

namespace rpa {

// The narrow path (rotary_dim not a multiple of 16): a warp a token, chunks of 4 or 2 bytes, its own sines, no
// row's loads ahead of another's. Calls body(u, turns, cs, head) for every unit u of `heads` heads of head_dim
// elements. (8191 tokens of 32 + 8 heads of 128: rotary_dim 24 61 us, 6 100 us, 128 on the other path 28.7.)
template <int VEC, typename F>
__device__ __forceinline__ void rope_units(const RopeTab& tab, int head_dim, int heads, int pos, F&& body) {
    const int lane = threadIdx.x & 31, units = head_dim / (2 * VEC);
    const int width = min(units, 32), heads_at_once = 32 / width;
    const int h0 = lane / width;
    if (h0 >= heads_at_once) return;
    for (int u = lane % width; u < units; u += width) {
        const bool turns = u * VEC < tab.rotary_dim / 2;
        float2 cs[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) cs[e] = turns ? rope_cos_sin(tab, u * VEC + e, pos) : make_float2(1.f, 0.f);
        for (int h = h0; h < heads; h += heads_at_once) body(u, turns, cs, h);
    }
}

// The rows of head h of token t: q's heads, then k's.
__device__ __forceinline__ const __nv_bfloat16* apply_in(const RopeApplyArgs& a, int t, int h) {
    const int hk = h - a.num_q_heads;
    return hk < 0 ? a.q.p + t * a.q.token + h * a.q.head : a.k.p + t * a.k.token + hk * a.k.head;
}
__device__ __forceinline__ __nv_bfloat16* apply_out(const RopeApplyArgs& a, int t, int h) {
    const int hk = h - a.num_q_heads;
    return hk < 0 ? a.q_out.p + t * a.q_out.token + h * a.q_out.head : a.k_out.p + t * a.k_out.token + hk * a.k_out.head;
}

// A unit's chunks turned in bf16.
template <bool INTER>
__device__ __forceinline__ void turn_chunks(uint4& xa, uint4& xb, const float4* cs, int stride) {
    float x[16];
    rope_unpack<8>(xa, x);
    rope_unpack<8>(xb, x + 8);
    rope_turn8<INTER>(cs, stride, x);
    xa = rope_pack<8>(x);
    xb = rope_pack<8>(x + 8);
}

template <bool INTER>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocksPerSm) rope_apply_kernel(const __grid_constant__ RopeApplyArgs a) {
    __shared__ RopeShared sh;
    const bool is_k = blockIdx.x >= a.q_share.blocks;
    const RopeRows& to = is_k ? a.k_out : a.q_out;
    rope_block<true, INTER>(
        a.tab, is_k ? a.k_share : a.q_share, is_k ? blockIdx.x - a.q_share.blocks : blockIdx.x, a.head_dim, a.num_tokens,
        is_k ? a.k : a.q, is_k ? a.num_k_heads : a.num_q_heads, sh,
        [&](int t0, int nt) {
            if (threadIdx.x < nt) sh.pos[threadIdx.x] = a.positions[t0 + threadIdx.x];
        },
        [&](int, int t, int h, bool turns, int ca, int cb, uint4 xa, uint4 xb, const float4* cs, int stride) {
            if (turns) turn_chunks<INTER>(xa, xb, cs, stride);
            __nv_bfloat16* dst = to.p + t * to.token + h * to.head;
            *reinterpret_cast<uint4*>(dst + ca) = xa;
            *reinterpret_cast<uint4*>(dst + cb) = xb;
        });
}

template <int VEC>
__global__ void __launch_bounds__(kRopeThreads) rope_apply_narrow_kernel(const __grid_constant__ RopeApplyArgs a) {
    using Chunk = typename RopeChunk<VEC>::type;
    const unsigned w = blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
    const int t = (int)w;
    if (w >= (unsigned)a.num_tokens) return;
    rope_units<VEC>(a.tab, a.head_dim, a.num_q_heads + a.num_k_heads, a.positions[t],
                    [&](int u, bool turns, const float2 (&cs)[VEC], int h) {
                        int ca, cb;
                        rope_chunks<VEC>(a.tab.rotary_dim, a.tab.interleaved, u, turns, ca, cb);
                        const __nv_bfloat16* src = apply_in(a, t, h);
                        Chunk xa = *reinterpret_cast<const Chunk*>(src + ca), xb = *reinterpret_cast<const Chunk*>(src + cb);
                        if (turns) {
                            float x[2 * VEC];
                            rope_unpack<VEC>(xa, x);
                            rope_unpack<VEC>(xb, x + VEC);
                            rope_turn<VEC>(a.tab.interleaved, cs, x);
                            xa = rope_pack<VEC>(x);
                            xb = rope_pack<VEC>(x + VEC);
                        }
                        __nv_bfloat16* dst = apply_out(a, t, h);
                        *reinterpret_cast<Chunk*>(dst + ca) = xa;
                        *reinterpret_cast<Chunk*>(dst + cb) = xb;
                    });
}

// The source row of head h of token t: q's heads, then k's, then v's.
__device__ __forceinline__ const __nv_bfloat16* update_in(const RopeUpdateArgs& a, int t, int h) {
    const int hk = h - a.num_q_heads, hv = hk - a.num_kv_heads;
    return hk < 0 ? a.q.p + t * a.q.token + h * a.q.head
                  : hv < 0 ? a.k.p + t * a.k.token + hk * a.k.head : a.v.p + t * a.v.token + hv * a.v.head;
}
// A unit's values to q_out or to the token's slot of the cache; turn(x) turns them (v turns nothing:
// its chunks are copied in the same order).
template <int VEC, int KV, typename Turn>
__device__ __forceinline__ void update_out(const RopeUpdateArgs& a, int t, int h, uint8_t* slot, bool turns, int ca, int cb,
                                           typename RopeChunk<VEC>::type xa, typename RopeChunk<VEC>::type xb, Turn&& turn) {
    using Chunk = typename RopeChunk<VEC>::type;
    const int hk = h - a.num_q_heads, hv = hk - a.num_kv_heads;
    const float inv = hv < 0 ? a.k_inv : a.v_inv;
    const bool convert = hk >= 0 && (KV != RPA_DTYPE_BF16 || inv != 1.f);
    turns = turns && hv < 0;
    uint8_t* cache = slot + (hv < 0 ? 2 * hk : 2 * hv + 1) * a.row_bytes;
    float x[2 * VEC];
    if (turns || convert) {
        rope_unpack<VEC>(xa, x);
        rope_unpack<VEC>(xb, x + VEC);
        if (turns) turn(x);
        if (convert) {
            rope_store_kv<KV, VEC>(cache, ca, x, inv);
            rope_store_kv<KV, VEC>(cache, cb, x + VEC, inv);
            return;
        }
        xa = rope_pack<VEC>(x);
        xb = rope_pack<VEC>(x + VEC);
    }
    __nv_bfloat16* dst = hk < 0 ? a.q_out + ((size_t)t * a.num_q_heads + h) * a.head_dim : reinterpret_cast<__nv_bfloat16*>(cache);
    *reinterpret_cast<Chunk*>(dst + ca) = xa;
    *reinterpret_cast<Chunk*>(dst + cb) = xb;
}

// At four blocks an SM a thread has 64 registers, and every form spills 40 to 120 bytes of them (three copies of
// the walk, with the slots' search in each). At three, without spills, 61 decodes and 2 x 1021 tokens of 16 + 8 +
// 8 heads of 256 take bf16 14.6, fp8 12.2, int8 13.2 and int4 13.3 us instead of 12.4, 12.3, 12.7 and 13.1; 4 x
// 4096 tokens 69, 64, 66 and 64 instead of 69, 62, 64 and 65.
template <bool INTER, int KV>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocksPerSm) rpa_rope_update_kernel(const __grid_constant__ RopeUpdateArgs a) {
    __shared__ RopeShared sh;
    // rpa_rope_forward_update's plan behind may start now: it reads only metadata this kernel does
    // not write, and it ends after this grid has
    pdl_launch_dependents();
    __shared__ int cu[kRopeCu];
    auto resolve = [&](int t0, int nt) {
        if (a.max_num_seqs < kRopeCu) {
            // all of cu_q_lens in one round trip, then a token a thread: two more for all of them (a warp a
            // token took four or five, again for every eight tokens: 4 x 4096 tokens 74.0 us, now 70.5)
            for (int i = threadIdx.x; i <= a.max_num_seqs; i += kRopeThreads) cu[i] = a.cu_q_lens[i];
            const int num = a.num_seqs[0];
            const bool some = num > 0 && num <= a.max_num_seqs;
            if (!some && num != 0 && t0 == 0 && threadIdx.x == 0) set_error(a.err, RPA_DEV_ERR_NUM_SEQS);
            __syncthreads();
            if (threadIdx.x < nt) {
                const int t = t0 + threadIdx.x;
                int pos = 0;
                uint8_t* slot = nullptr;
                if (some && cu[0] <= t) {
                    const int s = seq_of_token(cu, num, t);
                    const uint32_t bad = rope_slot_of(a, t, s, cu[s], cu[s + 1], cu[num], pos, slot);
                    if (bad) set_error(a.err, bad);
                }
                if (a.positions) pos = a.positions[t];
                sh.pos[threadIdx.x] = pos;
                sh.slot[threadIdx.x] = slot;
            }
            return;
        }
        for (int k = threadIdx.x >> 5; k < nt; k += kRopeWarps) {  // a warp a token
            int pos = 0;
            uint8_t* slot = nullptr;
            if (!rope_slot(a, t0 + k, pos, slot)) slot = nullptr;
            if (a.positions) pos = a.positions[t0 + k];
            if ((threadIdx.x & 31) == 0) {
                sh.pos[k] = pos;
                sh.slot[k] = slot;
            }
        }
    };
    unsigned share = blockIdx.x;
    if (share < a.q_share.blocks) {
        rope_block<true, INTER>(
            a.tab, a.q_share, share, a.head_dim, a.max_num_tokens, a.q, a.num_q_heads, sh, resolve,
            [&](int k, int t, int h, bool turns, int ca, int cb, uint4 xa, uint4 xb, const float4* cs, int stride) {
                if (!sh.slot[k]) return;
                if (turns) turn_chunks<INTER>(xa, xb, cs, stride);
                __nv_bfloat16* dst = a.q_out + ((size_t)t * a.num_q_heads + h) * a.head_dim;
                *reinterpret_cast<uint4*>(dst + ca) = xa;
                *reinterpret_cast<uint4*>(dst + cb) = xb;
            });
        return;
    }
    // a unit of k (part 0) or v (part 1) to the cache
    auto put = [&](int part, int k, int h, bool turns, int ca, int cb, uint4 xa, uint4 xb, const float4* cs, int stride, float inv) {
        uint8_t* slot = sh.slot[k];
        if (!slot) return;
        uint8_t* row = slot + (2 * h + part) * a.row_bytes;
        if (KV != RPA_DTYPE_BF16 || inv != 1.f) {
            float x[16];
            rope_unpack<8>(xa, x);
            rope_unpack<8>(xb, x + 8);
            if (turns) rope_turn8<INTER>(cs, stride, x);
            rope_store_kv<KV, 8>(row, ca, x, inv);
            rope_store_kv<KV, 8>(row, cb, x + 8, inv);
        } else {
            if (turns) turn_chunks<INTER>(xa, xb, cs, stride);
            *reinterpret_cast<uint4*>(row + 2 * ca) = xa;
            *reinterpret_cast<uint4*>(row + 2 * cb) = xb;
        }
    };
    share -= a.q_share.blocks;
    if (share < a.kv_share.blocks) {
        rope_block<true, INTER>(a.tab, a.kv_share, share, a.head_dim, a.max_num_tokens, a.k, a.num_kv_heads, sh, resolve,
                                [&](int k, int, int h, bool turns, int ca, int cb, uint4 xa, uint4 xb, const float4* cs, int stride) {
                                    put(0, k, h, turns, ca, cb, xa, xb, cs, stride, a.k_inv);
                                });
    } else {
        rope_block<false, INTER>(a.tab, a.kv_share, share - a.kv_share.blocks, a.head_dim, a.max_num_tokens, a.v,
                                 a.num_kv_heads, sh, resolve,
                                 [&](int k, int, int h, bool, int ca, int cb, uint4 xa, uint4 xb, const float4* cs, int stride) {
                                     put(1, k, h, false, ca, cb, xa, xb, cs, stride, a.v_inv);
                                 });
    }
}

template <int VEC, int KV>
__global__ void __launch_bounds__(kRopeThreads) rpa_rope_update_narrow_kernel(const __grid_constant__ RopeUpdateArgs a) {
    using Chunk = typename RopeChunk<VEC>::type;
    pdl_launch_dependents();  // as above
    const unsigned w = blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
    const int t = (int)w;
    if (w >= (unsigned)a.max_num_tokens) return;
    int pos;
    uint8_t* slot;
    if (!rope_slot(a, t, pos, slot)) return;
    if (a.positions) pos = a.positions[t];
    rope_units<VEC>(a.tab, a.head_dim, a.num_q_heads + 2 * a.num_kv_heads, pos,
                    [&](int u, bool turns, const float2 (&cs)[VEC], int h) {
                        int ca, cb;
                        rope_chunks<VEC>(a.tab.rotary_dim, a.tab.interleaved, u, turns, ca, cb);
                        const __nv_bfloat16* src = update_in(a, t, h);
                        update_out<VEC, KV>(a, t, h, slot, turns, ca, cb, *reinterpret_cast<const Chunk*>(src + ca),
                                            *reinterpret_cast<const Chunk*>(src + cb),
                                            [&](float (&x)[2 * VEC]) { rope_turn<VEC>(a.tab.interleaved, cs, x); });
                    });
}

constexpr int kRopePasses = 5, kRopeBlocks = 16;

// Elements per chunk: 16 bytes where the turned part's halves are whole chunks, else two elements
// or one.
static int rope_vec(const RopeTab& t) { return t.rotary_dim % 16 == 0 ? 8 : t.rotary_dim % 4 == 0 ? 2 : 1; }

// The shares of one kind, `share` head rows each or fewer.
static RopeShare rope_share(const RopeTab& tab, int tokens, int heads, int head_dim, double share) {
    const int rows = kRopeThreads / (head_dim / 16);  // head rows a block holds at once
    const int most = min(kRopeTokens, tab.rotary_dim ? kRopePairs / (tab.rotary_dim / 2) : kRopeTokens);
    RopeShare s = {1, heads, 1, 0};
    if (heads == 0) return s;
    s.tokens = max(1, min(most, (int)min(share / heads, 1e6)));
    s.parts = max(1, min(cdiv(heads, rows), (int)(heads / max(share, 1.0))));
    s.heads = cdiv(heads, s.parts);
    s.parts = cdiv(heads, s.heads);
    s.blocks = (unsigned)(((long long)tokens + s.tokens - 1) / s.tokens * s.parts);
    return s;
}

// Shares of both kinds: a's of ha heads, b's of hb, nb times.  A block finds its tokens' slots and sines
// before it can store, some 2 us, so it wants several passes over its threads (kRopePasses); more than
// kRopeBlocks blocks an SM only repeat that; and a small call is spread over every SM twice, by tokens and
// then by heads.
static void rope_shares(const RopeTab& tab, int tokens, int ha, int hb, int nb, int head_dim, int num_sms, RopeShare& a, RopeShare& b) {
    const double all = (double)tokens * (ha + nb * hb), passes = kRopePasses * (double)(kRopeThreads / (head_dim / 16));
    double share = min(max(passes, all / (kRopeBlocks * num_sms)), all / (2 * num_sms));
    // what the SMs hold at once and up to half as many again goes as one round of longer shares (a cache write of
    // 61 decodes and 2 x 1021 tokens of 32 heads of 256 15.9 us, in two rounds 17.7; of 2700 tokens of 48 heads of
    // 128 12.6 and 13.9, 2200 of them 11.3 and 11.1, 2000 of 32 heads of 256 11.9 and 11.4; rope_apply of 3000
    // tokens of 40 heads 11.1 and 11.5). Between one and a half and two and a half one round would gain 2 to 8 %
    // more, beyond it nothing (8191 tokens, either way the same)
    const int at_once = kRopeBlocksPerSm * num_sms;
    for (int i = 0; i < 40; ++i, share *= 1.03) {
        a = rope_share(tab, tokens, ha, head_dim, share);
        b = rope_share(tab, tokens, hb, head_dim, share);
        const double blocks = a.blocks + (double)nb * b.blocks;
        if (blocks <= at_once || blocks > 1.5 * at_once) break;
    }
}

// Blocks of kRopeWarps warps.
static unsigned rope_blocks(long long warps) { return (unsigned)((warps + kRopeWarps - 1) / kRopeWarps); }

cudaError_t launch_rope_apply(RopeApplyArgs& a, int num_sms, cudaStream_t stream) {
    ProfScope ps("rope_apply", stream);
    const int vec = rope_vec(a.tab);
    if (vec == 8) {
        rope_shares(a.tab, a.num_tokens, a.num_q_heads, a.num_k_heads, 1, a.head_dim, num_sms, a.q_share, a.k_share);
        const unsigned grid = a.q_share.blocks + a.k_share.blocks;
        if (a.tab.interleaved)
            rope_apply_kernel<true><<<grid, kRopeThreads, 0, stream>>>(a);
        else
            rope_apply_kernel<false><<<grid, kRopeThreads, 0, stream>>>(a);
    } else if (vec == 2) {
        rope_apply_narrow_kernel<2><<<rope_blocks(a.num_tokens), kRopeThreads, 0, stream>>>(a);
    } else {
        rope_apply_narrow_kernel<1><<<rope_blocks(a.num_tokens), kRopeThreads, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

template <int KV>
static cudaError_t launch_update_kv(RopeUpdateArgs& a, int num_sms, cudaStream_t stream) {
    const int vec = rope_vec(a.tab);
    if (vec == 8) {
        rope_shares(a.tab, a.max_num_tokens, a.num_q_heads, a.num_kv_heads, 2, a.head_dim, num_sms, a.q_share, a.kv_share);
        const unsigned grid = a.q_share.blocks + 2 * a.kv_share.blocks;
        if (a.tab.interleaved)
            rpa_rope_update_kernel<true, KV><<<grid, kRopeThreads, 0, stream>>>(a);
        else
            rpa_rope_update_kernel<false, KV><<<grid, kRopeThreads, 0, stream>>>(a);
    } else if (vec == 2) {
        rpa_rope_update_narrow_kernel<2, KV><<<rope_blocks(a.max_num_tokens), kRopeThreads, 0, stream>>>(a);
    } else {
        if constexpr (KV == RPA_DTYPE_INT4)
            return cudaErrorInvalidValue;  // (the host refuses it)
        else
            rpa_rope_update_narrow_kernel<1, KV><<<rope_blocks(a.max_num_tokens), kRopeThreads, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_rope_update(RopeUpdateArgs& a, int num_sms, cudaStream_t stream) {
    ProfScope ps("rpa_rope_update", stream);
    switch (a.kv_dtype) {
        case RPA_DTYPE_BF16: return launch_update_kv<RPA_DTYPE_BF16>(a, num_sms, stream);
        case RPA_DTYPE_FP8_E4M3: return launch_update_kv<RPA_DTYPE_FP8_E4M3>(a, num_sms, stream);
        case RPA_DTYPE_INT8: return launch_update_kv<RPA_DTYPE_INT8>(a, num_sms, stream);
        case RPA_DTYPE_INT4: return launch_update_kv<RPA_DTYPE_INT4>(a, num_sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace rpa
