"""Plain float64 forms of the rotary, appending and cross-attention operators, on CPU tensors."""
import math

import torch


def frequencies(rotary_dim, base=10000.0, scaling=None):
    """(angle per position of each pair, amplitude) from the definitions in include/rpa.h."""
    s = dict(scaling or {"type": "none"})
    kind, f, amp = s.pop("type"), [], s.get("attention_factor") or 1.0
    if kind == "yarn" and not s.get("attention_factor"):
        amp = 0.1 * math.log(s["factor"]) + 1.0
    if kind == "ntk":
        base = base * s["factor"] ** (rotary_dim / (rotary_dim - 2))

    def pair_at(turns):  # the (real) pair index that makes `turns` turns over the original context
        return rotary_dim * math.log(s["original_max_position"] / (2 * math.pi * turns)) / (2 * math.log(base))

    for i in range(rotary_dim // 2):
        w = base ** (-2.0 * i / rotary_dim)
        if kind == "linear":
            w /= s["factor"]
        elif kind == "llama3":
            n = s["original_max_position"] * w / (2 * math.pi)
            lo, hi = s["low_freq_factor"], s["high_freq_factor"]
            keep = 1.0 if n >= hi else 0.0 if n <= lo else (n - lo) / (hi - lo)
            w = keep * w + (1 - keep) * w / s["factor"]
        elif kind == "yarn":
            low = max(math.floor(pair_at(s.get("beta_fast", 32.0))), 0)
            high = min(math.ceil(pair_at(s.get("beta_slow", 1.0))), rotary_dim - 1)
            share = 0.0 if i < low else 1.0 if i >= high else (i - low) / (high - low)
            w = share * w / s["factor"] + (1 - share) * w
        f.append(w)
    return torch.tensor(f, dtype=torch.float64), amp


def rope(x, positions, freq, amp, interleaved, inverse=False):
    """x [T, heads, D] turned to positions [T], float64."""
    x = x.double()
    r = 2 * freq.numel()
    angle = positions.double()[:, None, None] * freq
    c, s = amp * angle.cos(), amp * angle.sin() * (-1.0 if inverse else 1.0)
    y = x.clone()
    i = torch.arange(r // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def rope_slack(x, freq, amp, interleaved):
    """How far float32 arithmetic may be from ``rope``: the angle over pi is rounded once (relative
    2^-24, so pi 2^-24 at most), sincospi is within 2 units in the last place of 1 (2 * 2^-24), the
    amplitude's factor, the product and the sum round once each (3 * 2^-24): 9 * 2^-24 < 2^-20 times
    amp (|x| + |y|); the other elements are exact."""
    x = x.double().abs()
    r = 2 * freq.numel()
    out = torch.zeros_like(x)
    i = torch.arange(r // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    out[..., a] = out[..., b] = (x[..., a] + x[..., b]) * abs(amp) * 2.0 ** -20
    return out


def half_step(v, dtype):
    """The largest rounding error of the value v in a storage type (e4m3 and integers saturate first)."""
    v = v.double().abs()
    if dtype == torch.bfloat16:
        return v * 2.0 ** -8 + 2.0 ** -134  # the second term: half a subnormal step
    if dtype == torch.float8_e4m3fn:
        return (v * 2.0 ** -4).clamp(min=2.0 ** -10)
    return torch.full_like(v, 0.5)


def unpack_int4(x):
    """uint8 [..., D / 2] -> int64 [..., D]: element 2i in the low nibble of byte i."""
    x = x.to(torch.int64)
    pair = torch.stack([x & 15, x >> 4], -1).flatten(-2)
    return torch.where(pair > 7, pair - 16, pair)


def stored_values(x):
    """A cache tensor's elements in float64 (unscaled)."""
    return unpack_int4(x).double() if x.dtype == torch.uint8 else x.double()


LIMITS = {torch.float8_e4m3fn: (-448.0, 448.0), torch.int8: (-128.0, 127.0), torch.uint8: (-8.0, 7.0)}


def attend_all(q, kv_pages, kv_lens, page_indices, cu_q_lens, num_seqs, *, sm_scale, soft_cap=None, k_scale=None,
               v_scale=None):
    """Every query of a sequence over all its keys, float64; rows of no sequence are NaN, a sequence
    without keys gives zeros.  Scaled caches are read as bf16(float(x) * scale)."""
    T, hq, d = q.shape
    out = torch.full((T, hq, d), math.nan, dtype=torch.float64)
    ps, hkv = kv_pages.shape[1], kv_pages.shape[2] // 2
    for s in range(num_seqs):
        a, b, n = int(cu_q_lens[s]), int(cu_q_lens[s + 1]), int(kv_lens[s])
        out[a:b] = 0.0
        if n == 0 or a == b:
            continue
        pages = page_indices[s, :-(-n // ps)].long()
        x = stored_values(kv_pages.view(torch.uint8)[pages].view(kv_pages.dtype)).flatten(0, 1)[:n]
        k, v = x[:, 0::2], x[:, 1::2]
        if k_scale or v_scale:
            k = (k.float() * (k_scale or 1.0)).bfloat16().double()
            v = (v.float() * (v_scale or 1.0)).bfloat16().double()
        k, v = (y.repeat_interleave(hq // hkv, dim=1) for y in (k, v))
        w = torch.einsum("qhd,khd->hqk", q[a:b].double(), k) * sm_scale
        if soft_cap:
            w = soft_cap * torch.tanh(w / soft_cap)
        out[a:b] = torch.einsum("hqk,khd->qhd", torch.softmax(w, -1), v)
    return out
