// Rotary positions (rope_apply) and the cache write that turns its keys (rpa_rope_update_kv_cache),
// for sm_103a.
//
// Both only move memory: a turned element costs two fused multiply-adds against four bytes.  One
// warp takes one token: its lanes stand for the units of a head (rope.cuh) and of the heads beside
// it, keep their sines and cosines, and walk over the token's heads.
#include "common.cuh"
#include "kernels.h"
#include "profile.h"
#include "rope.cuh"

namespace rpa {

constexpr int kRopeThreads = 256;

// Calls body(u, turns, cs, head) for every unit u of `heads` heads of head_dim elements, with the
// cosines and sines of the unit's pairs at `pos` where it turns.
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

template <int VEC>
__global__ void __launch_bounds__(kRopeThreads) rope_apply_kernel(const __grid_constant__ RopeApplyArgs a) {
    const int warps = gridDim.x * (kRopeThreads / 32);
    for (int t = blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5); t < a.num_tokens; t += warps) {
        const int pos = a.positions[t];
        rope_units<VEC>(a.tab, a.head_dim, a.num_q_heads + a.num_k_heads, pos,
                        [&](int u, bool turns, const float2 (&cs)[VEC], int h) {
                            const bool is_k = h >= a.num_q_heads;
                            const int hh = is_k ? h - a.num_q_heads : h;
                            const RopeRows &in = is_k ? a.k : a.q, &out = is_k ? a.k_out : a.q_out;
                            const __nv_bfloat16* src = in.p + t * in.token + hh * in.head;
                            __nv_bfloat16* dst = out.p + t * out.token + hh * out.head;
                            int ca, cb;
                            rope_chunks<VEC>(a.tab, u, turns, ca, cb);
                            float x[2 * VEC];
                            load_bf16<VEC>(src + ca, x);
                            load_bf16<VEC>(src + cb, x + VEC);
                            if (turns) rope_turn<VEC>(a.tab.interleaved, cs, x);
                            store_bf16<VEC>(dst + ca, x);
                            store_bf16<VEC>(dst + cb, x + VEC);
                        });
    }
}

template <int VEC, int KV>
__global__ void __launch_bounds__(kRopeThreads) rpa_rope_update_kernel(const __grid_constant__ RopeUpdateArgs a) {
    const int warps = gridDim.x * (kRopeThreads / 32);
    // an rpa_forward plan kernel behind may start now: it reads only metadata this kernel does
    // not write, and it ends after this grid has
    pdl_launch_dependents();
    int num = a.num_seqs[0];
    if (num < 0 || num > a.max_num_seqs) {
        if (blockIdx.x == 0 && threadIdx.x == 0) set_error(a.err, RPA_DEV_ERR_NUM_SEQS);
        return;
    }
    const int hq = a.num_q_heads, hkv = a.num_kv_heads;
    for (int t = blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5); t < a.max_num_tokens; t += warps) {
        int pos;
        size_t slot;
        if (!rope_slot(a, num, t, pos, slot)) continue;
        if (a.positions) pos = a.positions[t];
        rope_units<VEC>(a.tab, a.head_dim, hq + 2 * hkv, pos,
                        [&](int u, bool turns, const float2 (&cs)[VEC], int h) {
                            const int kind = h < hq ? 0 : h < hq + hkv ? 1 : 2;  // q, k, v
                            const int hh = kind == 0 ? h : kind == 1 ? h - hq : h - hq - hkv;
                            const RopeRows& in = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
                            const __nv_bfloat16* src = in.p + t * in.token + hh * in.head;
                            int ca, cb;
                            rope_chunks<VEC>(a.tab, u, turns && kind < 2, ca, cb);
                            float x[2 * VEC];
                            load_bf16<VEC>(src + ca, x);
                            load_bf16<VEC>(src + cb, x + VEC);
                            if (turns && kind < 2) rope_turn<VEC>(a.tab.interleaved, cs, x);
                            if (kind == 0) {
                                __nv_bfloat16* dst = a.q_out + ((size_t)t * hq + hh) * a.head_dim;
                                store_bf16<VEC>(dst + ca, x);
                                store_bf16<VEC>(dst + cb, x + VEC);
                            } else {
                                uint8_t* row = static_cast<uint8_t*>(a.kv_pages) +
                                               (slot * 2 * hkv + 2 * hh + (kind - 1)) * (size_t)a.row_bytes;
                                const float inv = kind == 1 ? a.k_inv : a.v_inv;
                                store_kv<KV, VEC>(row, ca, x, inv);
                                store_kv<KV, VEC>(row, cb, x + VEC, inv);
                            }
                        });
    }
}

// Pairs per unit: 2 where the turned part's halves start on even elements.
static int rope_vec(const RopeTab& t) { return t.rotary_dim % 4 == 0 ? 2 : 1; }

static int rope_grid(int tokens, int num_sms) {
    return min(cdiv(tokens, kRopeThreads / 32), num_sms * (2048 / kRopeThreads));
}

cudaError_t launch_rope_apply(const RopeApplyArgs& a, int num_sms, cudaStream_t stream) {
    if (a.num_tokens <= 0) return cudaSuccess;
    ProfScope ps("rope_apply", stream);
    const int grid = rope_grid(a.num_tokens, num_sms);
    if (rope_vec(a.tab) == 2)
        rope_apply_kernel<2><<<grid, kRopeThreads, 0, stream>>>(a);
    else
        rope_apply_kernel<1><<<grid, kRopeThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <int KV>
static cudaError_t launch_update_kv(const RopeUpdateArgs& a, int num_sms, cudaStream_t stream) {
    const int grid = rope_grid(a.max_num_tokens, num_sms);
    if (rope_vec(a.tab) == 2) {
        rpa_rope_update_kernel<2, KV><<<grid, kRopeThreads, 0, stream>>>(a);
    } else {
        if constexpr (KV == RPA_DTYPE_INT4)
            return cudaErrorInvalidValue;  // (the host refuses it)
        else
            rpa_rope_update_kernel<1, KV><<<grid, kRopeThreads, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_rope_update(const RopeUpdateArgs& a, int num_sms, cudaStream_t stream) {
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
