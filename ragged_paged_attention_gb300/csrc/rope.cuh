// Rotary positions: the device code that rope_apply, the appending cache write and the fused
// plan share.
//
// Work is cut into units of 2 * VEC elements of one head, which hold VEC whole pairs: for the
// half pairing the chunks [u VEC, u VEC + VEC) and the same rotary_dim / 2 further on, for the
// interleaved one 2 VEC adjacent elements; past rotary_dim, 2 VEC adjacent elements that are
// copied.  Unit u's pairs are u VEC .. u VEC + VEC - 1 either way, so a thread that keeps its u
// keeps its sines and cosines from head to head.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace rpa {

// cos and sin of pair i at `pos`, times the amplitude.  pos * step modulo 2^64 is the fraction of
// a turn as a signed 64-bit number, exactly; its float32 value (relative error 2^-24) times 2^-63
// is the angle over pi.
__device__ __forceinline__ float2 rope_cos_sin(const RopeTab& t, int i, int pos) {
    const long long turn = (long long)((unsigned long long)(long long)pos * t.step[i]);
    float s, c;
    sincospif((float)turn * 0x1p-63f, &s, &c);
    return make_float2(c * t.amplitude, s * t.sin_amplitude);
}

// Element offsets in a head row of unit u's chunks a and b (VEC elements each).
template <int VEC>
__device__ __forceinline__ void rope_chunks(const RopeTab& t, int u, bool turns, int& a, int& b) {
    const bool half = turns && !t.interleaved;
    a = half ? u * VEC : 2 * u * VEC;
    b = half ? a + t.rotary_dim / 2 : a + VEC;
}

// The unit's 2 VEC values in place: x = chunk a then chunk b.
template <int VEC>
__device__ __forceinline__ void rope_turn(bool interleaved, const float2 (&cs)[VEC], float (&x)[2 * VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const int i = interleaved ? 2 * e : e, j = interleaved ? 2 * e + 1 : VEC + e;
        const float p = x[i], q = x[j];
        x[i] = fmaf(p, cs[e].x, -q * cs[e].y);
        x[j] = fmaf(q, cs[e].x, p * cs[e].y);
    }
}

template <int VEC>
__device__ __forceinline__ void load_bf16(const __nv_bfloat16* src, float* x) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = __bfloat162float(src[e]);
}
template <int VEC>
__device__ __forceinline__ void store_bf16(__nv_bfloat16* dst, const float* x) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) dst[e] = __float2bfloat16_rn(x[e]);
}

__device__ __forceinline__ int quant_int(float x, int lo, int hi) {
    return min(max(__float2int_rn(x), lo), hi);  // NaN converts to 0, values past int to its ends
}

// VEC values to the cache at element `at` of a head row, divided by the scale and rounded once.
template <int KV, int VEC>
__device__ __forceinline__ void store_kv(uint8_t* row, int at, const float* x, float inv) {
    if constexpr (KV == RPA_DTYPE_BF16) {
        __nv_bfloat16* d = reinterpret_cast<__nv_bfloat16*>(row) + at;
#pragma unroll
        for (int e = 0; e < VEC; ++e) d[e] = __float2bfloat16_rn(x[e] * inv);
    } else if constexpr (KV == RPA_DTYPE_FP8_E4M3) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) row[at + e] = __nv_cvt_float_to_fp8(x[e] * inv, __NV_SATFINITE, __NV_E4M3);
    } else if constexpr (KV == RPA_DTYPE_INT8) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) row[at + e] = (uint8_t)quant_int(x[e] * inv, -128, 127);
    } else {
        static_assert(VEC % 2 == 0 || KV != RPA_DTYPE_INT4, "int4 values are written two to a byte");
#pragma unroll
        for (int e = 0; e < VEC; e += 2)
            row[(at + e) / 2] = (uint8_t)((quant_int(x[e] * inv, -8, 7) & 15) | (quant_int(x[e + 1] * inv, -8, 7) << 4));
    }
}

// The slot of token t: its sequence, checked as the plan checks it.  False where the token is
// padding or its metadata is bad (the error word then says so).
__device__ __forceinline__ bool rope_slot(const RopeUpdateArgs& a, int num, int t, int& pos, size_t& slot) {
    if (num <= 0) return false;
    if (t >= a.cu_q_lens[num]) return false;  // padding
    const int s = seq_of_token(a.cu_q_lens, num, t);
    const int c0 = a.cu_q_lens[s], c1 = a.cu_q_lens[s + 1], ql = c1 - c0, kl = a.kv_lens[s];
    if (s == 0 && t < c0) return false;
    uint32_t bad = 0;
    if (c0 < 0 || t < c0 || t >= c1 || c1 > a.max_num_tokens)
        bad = RPA_DEV_ERR_TOKENS;
    else if (ql > kl)
        bad = RPA_DEV_ERR_Q_LEN;
    else if ((kl - 1) / a.page_size >= a.pages_per_seq)
        bad = RPA_DEV_ERR_KV_LEN;
    int page = 0;
    if (!bad) {
        pos = kl - ql + (t - c0);
        page = a.page_indices[(size_t)s * a.pages_per_seq + pos / a.page_size];
        if ((unsigned)page >= (unsigned)a.total_num_pages) bad = RPA_DEV_ERR_PAGE;
    }
    if (bad) {
        if ((threadIdx.x & 31) == 0) set_error(a.err, bad);
        return false;
    }
    slot = (size_t)page * a.page_size + pos % a.page_size;
    return true;
}

}  // namespace rpa
