// Rotary positions: the device code that rope_apply and the appending cache write share.
//
// Work is cut into units of 2 * VEC elements of one head, which hold VEC whole pairs: for the
// half pairing the chunks [u VEC, u VEC + VEC) and the same rotary_dim / 2 further on, for the
// interleaved one 2 VEC adjacent elements; past rotary_dim, 2 VEC adjacent elements that are
// copied.  Unit u's pairs are u VEC .. u VEC + VEC - 1 either way, so a lane that keeps its u
// keeps its sines and cosines from head to head.  VEC is 8 (16-byte chunks) where 16 divides
// rotary_dim, else 2 or 1.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace rpa {

// cos and sin of pair i at `pos`, times the amplitude.  pos * step modulo 2^64 is the fraction of
// a turn as a signed 64-bit number, exactly.  Its upper 24 bits are an exact float32, whose sine
// and cosine sincospi takes; the angle d of the 32 bits below (at most pi 2^-23; the last 8 bits
// are under 2^-55) turns them on by cos - d sin, sin + d cos (d^2 / 2 < 2^-43).  So the angle
// costs no precision: what is left is sincospi's own error and one rounding.
__device__ __forceinline__ float2 rope_cos_sin(const RopeTab& t, int i, int pos) {
    const unsigned long long turn = (unsigned long long)(long long)pos * t.step[i];
    const float hi = (float)((int)(turn >> 32) >> 8) * 0x1p-23f;
    const float d = (float)(uint32_t)(turn >> 8) * (0x1p-55f * 3.14159265358979f);
    float s, c;
    sincospif(hi, &s, &c);
    return make_float2(fmaf(-d, s, c) * t.amplitude, fmaf(d, c, s) * t.sin_amplitude);
}

// Element offsets in a head row of unit u's chunks a and b (VEC elements each).
template <int VEC>
__device__ __forceinline__ void rope_chunks(int rotary_dim, bool interleaved, int u, bool turns, int& a, int& b) {
    const bool half = turns && !interleaved;
    a = half ? u * VEC : 2 * u * VEC;
    b = half ? a + rotary_dim / 2 : a + VEC;
}

// The unit's 2 VEC values in place: x = chunk a then chunk b.
template <int VEC>
__device__ __forceinline__ void rope_turn(bool interleaved, const float2 (&cs)[VEC], float (&x)[2 * VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        float &p = interleaved ? x[2 * e] : x[e], &q = interleaved ? x[2 * e + 1] : x[VEC + e];
        const float y = fmaf(p, cs[e].x, -q * cs[e].y);
        q = fmaf(q, cs[e].x, p * cs[e].y);
        p = y;
    }
}

// ---- chunks of VEC bf16 elements as they lie in memory ----
template <int VEC>
struct RopeChunk;
template <>
struct RopeChunk<8> {
    using type = uint4;
};
template <>
struct RopeChunk<2> {
    using type = uint32_t;
};
template <>
struct RopeChunk<1> {
    using type = uint16_t;
};

template <int VEC>
__device__ __forceinline__ void rope_unpack(const typename RopeChunk<VEC>::type& c, float* x) {
    if constexpr (VEC == 1) {
        x[0] = __uint_as_float((uint32_t)c << 16);
    } else {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&c);
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
            x[2 * e] = __uint_as_float(w[e] << 16);
            x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
    }
}
template <int VEC>
__device__ __forceinline__ typename RopeChunk<VEC>::type rope_pack(const float* x) {
    typename RopeChunk<VEC>::type c;
    if constexpr (VEC == 1) {
        c = __bfloat16_as_ushort(__float2bfloat16_rn(x[0]));
    } else {
        uint32_t* w = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) w[e] = pack_bf16(x[2 * e], x[2 * e + 1]);
    }
    return c;
}

__device__ __forceinline__ int quant_int(float x, int lo, int hi) {
    return min(max(__float2int_rn(x), lo), hi);  // NaN converts to 0, values past int to its ends
}
// Two values as e4m3 bytes, the first in the low byte (nearest even, +-448 at most, NaN kept).
__device__ __forceinline__ uint32_t quant_e4m3x2(float x, float y) {
    return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}

// VEC values times the scale's float32 reciprocal, rounded to the cache's type, at element `at` of a head row.
// (A power of two's reciprocal is exact; with another scale the product is up to 2^-23 of itself off the quotient,
// a division, which takes several instructions an element, 2^-24.)
template <int KV, int VEC>
__device__ __forceinline__ void rope_store_kv(uint8_t* row, int at, const float* x, float inv) {
    float y[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) y[e] = x[e] * inv;
    if constexpr (KV == RPA_DTYPE_BF16) {
        *reinterpret_cast<typename RopeChunk<VEC>::type*>(row + 2 * at) = rope_pack<VEC>(y);
    } else if constexpr (KV == RPA_DTYPE_INT4) {
        static_assert(VEC % 2 == 0, "int4 values are written two to a byte");
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < VEC; ++e) w |= (uint32_t)(quant_int(y[e], -8, 7) & 15) << (4 * e);
        if constexpr (VEC == 8)
            *reinterpret_cast<uint32_t*>(row + at / 2) = w;
        else
            row[at / 2] = (uint8_t)w;
    } else {
        constexpr bool F8 = KV == RPA_DTYPE_FP8_E4M3;
        if constexpr (VEC == 1) {
            row[at] = (uint8_t)(F8 ? quant_e4m3x2(y[0], 0.f) : (uint32_t)quant_int(y[0], -128, 127));
        } else {
            uint32_t w[(VEC + 3) / 4] = {};
#pragma unroll
            for (int e = 0; e < VEC; e += 2) {
                const uint32_t two = F8 ? quant_e4m3x2(y[e], y[e + 1])
                                        : (uint32_t)(quant_int(y[e], -128, 127) & 255) | (uint32_t)(quant_int(y[e + 1], -128, 127) & 255) << 8;
                w[e / 4] |= (two & 0xffffu) << (8 * (e & 2));
            }
            if constexpr (VEC == 8)
                *reinterpret_cast<uint2*>(row + at) = make_uint2(w[0], w[1]);
            else
                *reinterpret_cast<uint16_t*>(row + at) = (uint16_t)w[0];
        }
    }
}

// The cache rows of token t's slot in sequence s, which has the queries [c0, c1) of `end`: the error bits
// that its metadata sets, checked as the plan checks it, and `slot` NULL then or where t is padding.
__device__ __forceinline__ uint32_t rope_slot_of(const RopeUpdateArgs& a, int t, int s, int c0, int c1, int end, int& pos,
                                                 uint8_t*& slot) {
    slot = nullptr;
    const int kl = a.kv_lens[s];
    if (t >= end) return 0;  // padding
    if (c0 < 0 || t < c0 || t >= c1 || c1 > a.max_num_tokens) return RPA_DEV_ERR_TOKENS;
    if (c1 - c0 > kl) return RPA_DEV_ERR_Q_LEN;
    if ((kl - 1) / a.page_size >= a.pages_per_seq) return RPA_DEV_ERR_KV_LEN;
    pos = kl - (c1 - t);
    const int page = a.page_indices[(size_t)s * a.pages_per_seq + pos / a.page_size];
    if ((unsigned)page >= (unsigned)a.total_num_pages) return RPA_DEV_ERR_PAGE;
    slot = static_cast<uint8_t*>(a.kv_pages) + ((size_t)page * a.page_size + pos % a.page_size) * 2 * a.num_kv_heads * a.row_bytes;
    return 0;
}

// The cache rows of token t's slot, found by the whole warp.  False where the token is padding or its
// metadata is bad (the error word then says so).  The sequence is found 32 entries of cu_q_lens at a time;
// the first 32, the count and the checks' values are each one round trip for a batch of up to 31 sequences.
__device__ __forceinline__ bool rope_slot(const RopeUpdateArgs& a, int t, int& pos, uint8_t*& slot) {
    const int lane = threadIdx.x & 31;
    const int first = a.cu_q_lens[min(lane, a.max_num_seqs)];  // (max_num_seqs + 1 entries, whatever num_seqs)
    const int num = a.num_seqs[0];
    if (num <= 0 || num > a.max_num_seqs) {
        if (num != 0 && t == 0 && lane == 0) set_error(a.err, RPA_DEV_ERR_NUM_SEQS);
        return false;
    }
    int s = 0, left = num;  // the sequence is among [s, s + left)
    for (bool fresh = true; fresh || left > 1; fresh = false) {
        const int stride = cdiv(left, 32), i = lane * stride;
        const int v = fresh && stride == 1 ? first : i < left ? a.cu_q_lens[s + i] : 0;
        const int upto = __popc(__ballot_sync(0xffffffffu, i < left && v <= t));
        if (upto == 0) return false;  // before the first sequence
        s += (upto - 1) * stride;
        left = min(stride, left - (upto - 1) * stride);
    }
    const uint32_t bad = rope_slot_of(a, t, s, a.cu_q_lens[s], a.cu_q_lens[s + 1], a.cu_q_lens[num], pos, slot);
    if (bad && lane == 0) set_error(a.err, bad);
    return slot != nullptr;
}

// Positions and slots (NULL where the token has none) of the block's tokens t0 .. t0 + nt - 1, by the whole block;
// cu: kRopeCu ints of shared memory.  Behind it a barrier.
constexpr int kRopeCu = 1024;
constexpr int kRopeTokens = 32;     // most tokens of a block
template <int kThreads>
__device__ __forceinline__ void rope_slots(const RopeUpdateArgs& a, int t0, int nt, int* cu, int* pos_of, uint8_t** slot_of) {
    if (a.max_num_seqs < kRopeCu) {
        // all of cu_q_lens in one round trip, then a token a thread: two more for all of them (a warp a
        // token took four or five, again for every eight tokens: 4 x 4096 tokens 74.0 us, now 70.5)
        for (int i = threadIdx.x; i <= a.max_num_seqs; i += kThreads) cu[i] = a.cu_q_lens[i];
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
            pos_of[threadIdx.x] = pos;
            slot_of[threadIdx.x] = slot;
        }
        return;
    }
    for (int k = threadIdx.x >> 5; k < nt; k += kThreads / 32) {  // a warp a token
        int pos = 0;
        uint8_t* slot = nullptr;
        if (!rope_slot(a, t0 + k, pos, slot)) slot = nullptr;
        if (a.positions) pos = a.positions[t0 + k];
        if ((threadIdx.x & 31) == 0) {
            pos_of[k] = pos;
            slot_of[k] = slot;
        }
    }
}

// ---- a block's walk over head rows: the 16-byte path ----
// A block takes head rows of one kind (q, k or v): of whole tokens, or of a part of one token's
// heads.  Its threads stand for the units of as many rows as they hold (256 / units) and walk down
// the share with the loads of kRopeAhead rows in flight, the first of them issued before anything
// else.  The tokens' positions are found and their sines and cosines computed once a block, one or a
// few a thread, and read back from shared memory by the units.
constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopeBlocksPerSm = 4;
constexpr int kRopeAhead = 3;
constexpr int kRopePairs = 2048;    // most pairs whose sines a block keeps (16 KB)

struct RopeShared {
    // pairs 8 u + 2 j and 8 u + 2 j + 1 of token k at [(4 k + j) * rotary_dim / 16 + u] as
    // (cos, cos, sin, sin): the lanes of one head read adjacent 16-byte words
    float4 cs[kRopePairs / 2];
    uint8_t* slot[kRopeTokens];
    int pos[kRopeTokens];
};

// The unit's 16 values turned, two pairs an instruction; cs: its words of RopeShared::cs, `stride`
// apart.
template <bool INTER>
__device__ __forceinline__ void rope_turn8(const float4* cs, int stride, float (&x)[16]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 v = cs[j * stride];
        const float2 c = make_float2(v.x, v.y), s = make_float2(v.z, v.w), ns = make_float2(-v.z, -v.w);
        const int p0 = INTER ? 4 * j : 2 * j, p1 = INTER ? p0 + 2 : p0 + 1, q0 = INTER ? p0 + 1 : 8 + p0, q1 = INTER ? p0 + 3 : q0 + 1;
        const float2 p = make_float2(x[p0], x[p1]), q = make_float2(x[q0], x[q1]);
        const float2 y = ffma2(q, ns, fmul2(p, c)), z = ffma2(q, c, fmul2(p, s));
        x[p0] = y.x;
        x[p1] = y.y;
        x[q0] = z.x;
        x[q1] = z.y;
    }
}

// Share `share` of the kind's rows `in`, whose tokens have `heads` heads.  resolve(t0, n) writes the n
// tokens' positions into sh.pos (and what out needs of them); out(k, t, h, turns, ca, cb, xa, xb, cs, stride)
// takes a unit of head h of the block's k-th token t: its element offsets, its chunks as loaded and
// where its sines and cosines are (rope_turn8's arguments).
template <bool TURN, bool INTER, typename Resolve, typename Out>
__device__ __forceinline__ void rope_block(const RopeTab& tab, const RopeShare& split, unsigned share, int head_dim,
                                           int num_tokens, const RopeRows& in, int heads, RopeShared& sh, Resolve&& resolve,
                                           Out&& out) {
    const int tid = threadIdx.x, units = head_dim / 16, rows = kRopeThreads / units;
    const int u = tid % units, row0 = tid / units;
    const unsigned span = share / (unsigned)split.parts;
    const int h0 = (int)(share - span * split.parts) * split.heads, nh = min(split.heads, heads - h0);
    const int t0 = (int)(span * split.tokens), nt = min(split.tokens, num_tokens - t0);
    const bool turns = TURN && u * 16 < tab.rotary_dim;
    int ca, cb;
    rope_chunks<8>(tab.rotary_dim, INTER, u, turns, ca, cb);
    // rows of this thread: row0, row0 + rows, ..; each as token k of the block and its head h (from h0)
    const int dk = rows / nh, dh = rows - dk * nh;
    int k = row0 / nh, h = row0 - k * nh;
    if (row0 >= rows) k = nt;  // (threads past the last whole row have none)
    int k_next = k, h_next = h;
    const __nv_bfloat16* src = in.p + (t0 + (long long)k) * in.token + (h0 + h) * in.head + ca;
    const long long step = dk * in.token + dh * in.head, wrap = in.token - nh * in.head;
    uint4 xa[kRopeAhead], xb[kRopeAhead];
    auto load = [&](int j) {
        if (k_next < nt) {
            xa[j] = *reinterpret_cast<const uint4*>(src);
            xb[j] = *reinterpret_cast<const uint4*>(src + (cb - ca));
        }
        k_next += dk;
        h_next += dh;
        src += step;
        if (h_next >= nh) {
            h_next -= nh;
            ++k_next;
            src += wrap;
        }
    };
#pragma unroll
    for (int j = 0; j < kRopeAhead; ++j) load(j);
    resolve(t0, nt);
    __syncthreads();
    const int turning = tab.rotary_dim / 16;  // units that turn
    if (TURN) {
        const int pairs = tab.rotary_dim / 2;
        for (int i = tid; i < nt * pairs; i += kRopeThreads) {
            const int tok = i / pairs, pair = i - tok * pairs;
            const float2 v = rope_cos_sin(tab, pair, sh.pos[tok]);
            float* at = reinterpret_cast<float*>(&sh.cs[(4 * tok + ((pair & 7) >> 1)) * turning + (pair >> 3)]) + (pair & 1);
            at[0] = v.x;
            at[2] = v.y;
        }
        __syncthreads();
    }
    while (k < nt) {
#pragma unroll
        for (int j = 0; j < kRopeAhead; ++j) {
            if (k >= nt) break;
            out(k, t0 + k, h0 + h, turns, ca, cb, xa[j], xb[j], sh.cs + 4 * k * turning + u, turning);
            k += dk;
            h += dh;
            if (h >= nh) {
                h -= nh;
                ++k;
            }
            load(j);
        }
    }
}

}  // namespace rpa
