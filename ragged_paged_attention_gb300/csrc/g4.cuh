// Rows of the 4-bit cache (RPA_DTYPE_G4): a token's K and V of one KV head.
//
//   [ K: D / 2 bytes | V: D / 2 bytes | K's groups: (s, m) bf16 pairs | V's groups ]
//
// Element 2i of a part is the low half of its byte i.  x = s n + m with n in 0..15, m a group's least
// value and s the step.  A group is 64 elements, or 32 at head_dim 64: a row then fills whole 16-byte
// units (80, 144 and 288 bytes), which bulk copies move, and two groups at least keep a part's own
// scales apart.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace rpa {

template <int D>
struct G4 {
    static_assert(D == 64 || D == 128 || D == 256, "head_dim");
    static constexpr int kGroup = D == 64 ? 32 : 64;
    static constexpr int NG = D / kGroup;          // groups of K (and of V)
    static constexpr int kPart = D / 2;            // bytes of K's (or V's) values
    static constexpr int kParams = D;              // offset of the (s, m) pairs: K's, then V's
    static constexpr int kRow = D + 8 * NG;        // bytes of a row
};

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint4& v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The greater and the lesser of bf16 pairs; a NaN stays one.
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t bf16x2_min(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// ---- writing ----
// (greatest, -least) of a chunk of 8 values, one bf16 each.
__device__ __forceinline__ uint32_t g4_extremes(const uint4& x) {
    const uint32_t mx = bf16x2_max(bf16x2_max(x.x, x.y), bf16x2_max(x.z, x.w));
    const uint32_t mn = bf16x2_min(bf16x2_min(x.x, x.y), bf16x2_min(x.z, x.w)) ^ 0x80008000u;
    return bf16x2_max(__byte_perm(mx, mn, 0x5410), __byte_perm(mx, mn, 0x7632));
}
// What is held is finite: NaN counts as 0, and all else lies within +-2^48, so that the attention kernels can
// move its exponents by what their tensor operands need. (A chunk's extremes tell whether it has any such value.)
__device__ __forceinline__ void g4_limit(uint4& x, uint32_t& extremes) {
    if (fabsf(bf16_lo(extremes)) <= 0x1p48f && fabsf(bf16_hi(extremes)) <= 0x1p48f) return;
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t lo = (w[e] & 0x7fffu) > 0x7f80u ? 0u : w[e] & 0xffffu, hi = (w[e] & 0x7fff0000u) > 0x7f800000u ? 0u : w[e] & 0xffff0000u;
        w[e] = bf16x2_min(bf16x2_max(lo | hi, 0xd780d780u), 0x57805780u);
    }
    x = make_uint4(w[0], w[1], w[2], w[3]);
    extremes = g4_extremes(x);
}
// The group's (s, m) from its extremes.
__device__ __forceinline__ uint32_t g4_params(uint32_t extremes) {
    const float hi = bf16_lo(extremes), m = -bf16_hi(extremes);
    return pack_bf16(__fdiv_rn(hi - m, 15.f), m);
}
// 8 values -> their 4-bit numbers, two a byte.  bf16 data often lie in the middle between two numbers, where the product
// with s's float32 reciprocal would fall on either side.  The reciprocal as a sum of two floats (Brisebarre and
// Muller, "Correctly rounded multiplication by arbitrary precision constants", 2008) gives a quotient within 2^-46 of
// itself before its one rounding, so one that is a float comes out exactly: 16 instructions a pair of values became 10 (4 x
// 4096 tokens of 32 + 8 + 8 heads of 128: 97 us, with divisions 137; 87 now in a graph).  Adding 2^23 then rounds to nearest even, and leaves the
// number in the low bits.
__device__ __forceinline__ uint32_t g4_numbers(const uint4& x, uint32_t sm) {
    const float s = bf16_lo(sm), m = bf16_hi(sm);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t r = 0;
    if (s >= 0x1p-100f) {
        const float r1 = __frcp_rn(s), r2 = fmaf(-r1, s, 1.f) * r1;
        const float2 nm = make_float2(-m, -m), rr1 = make_float2(r1, r1), rr2 = make_float2(r2, r2), up = make_float2(0x1p23f, 0x1p23f);
        // (each sum's bits are those of 2^23 plus the number)
        constexpr uint32_t kUp = 0x4b000000u;
        uint32_t off = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 d = fadd2(make_float2(bf16_lo(w[e]), bf16_hi(w[e])), nm);
            float2 t = ffma2(d, rr1, fmul2(d, rr2));
            t = fadd2(make_float2(fminf(t.x, 15.f), fminf(t.y, 15.f)), up);
            r += __float_as_uint(t.x) << (8 * e);
            r += __float_as_uint(t.y) << (8 * e + 4);
            off += (kUp << (8 * e)) + (kUp << (8 * e + 4));
        }
        return r - off;
    }
    const float by = s > 0.f ? s : INFINITY;  // (steps next to nothing, and none)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        r |= (uint32_t)min(__float2int_rn(__fdiv_rn(bf16_lo(w[e]) - m, by)), 15) << (8 * e);
        r |= (uint32_t)min(__float2int_rn(__fdiv_rn(bf16_hi(w[e]) - m, by)), 15) << (8 * e + 4);
    }
    return r;
}
// A thread's 16 elements (chunks of 8 at ca and cb) of a head's K or V into its row, by the head_dim / 16
// adjacent lanes that hold the head between them.
__device__ __forceinline__ void g4_store_unit(uint8_t* row, int part, int head_dim, int ca, int cb, uint4 xa, uint4 xb) {
    const int units = head_dim / 16, lane = threadIdx.x & 31, u = lane & (units - 1);
    const int lg = head_dim == 64 ? 5 : 6, groups = head_dim >> lg, ga = ca >> lg, gb = cb >> lg;
    const uint32_t lanes = ((1u << units) - 1) << (lane - u);
    uint32_t ea = g4_extremes(xa), eb = g4_extremes(xb);
    g4_limit(xa, ea);
    g4_limit(xb, eb);
    uint32_t sa = 0, sb = 0, mine = 0;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        if (g >= groups) break;
        uint32_t v = 0xff80ff80u;  // (-inf, -inf)
        if (ga == g) v = ea;
        if (gb == g) v = bf16x2_max(v, eb);
        for (int o = units / 2; o > 0; o >>= 1) v = bf16x2_max(v, __shfl_xor_sync(lanes, v, o));
        v = g4_params(v);
        if (ga == g) sa = v;
        if (gb == g) sb = v;
        if (u == g) mine = v;
    }
    *reinterpret_cast<uint32_t*>(row + part * (head_dim / 2) + ca / 2) = g4_numbers(xa, sa);
    *reinterpret_cast<uint32_t*>(row + part * (head_dim / 2) + cb / 2) = g4_numbers(xb, sb);
    if (u < groups) *reinterpret_cast<uint32_t*>(row + head_dim + 4 * (part * groups + u)) = mine;
}

// ---- reading ----
// 8 numbers -> the bf16 nearest to s n + m, in order.
__device__ __forceinline__ uint4 g4_values8(uint32_t w, float s, float m) {
    uint32_t r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        r[e] = pack_bf16(fmaf((float)(w >> (8 * e) & 15), s, m), fmaf((float)(w >> (8 * e + 4) & 15), s, m));
    return make_uint4(r[0], r[1], r[2], r[3]);
}

}  // namespace rpa
