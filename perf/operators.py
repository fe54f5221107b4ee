"""Cases of the positional, appending and cross-attention operators, with their plain forms.

``rope``    rotary positions on packed q and k (``api.rope_apply``)
``append``  new K/V rows to their pages, rotated (and rounded to the cache's type) on the way,
            q rotated beside them (``api.rpa_rope_update_kv_cache``)
``cross``   attention of every query to all of its sequence's cached keys, as a decoder attends
            to an encoder's states (``api.rpa_cross_forward``)
``step``    append, then causal attention over the cache, in one call
            (``api.rpa_rope_forward_update``)

With ``own`` false ``run`` computes them from elementary torch operations in float32 (angles in
float64); ``exact`` restates them in float64.
"""
import math
import random

import numpy as np
import torch

own = False

LLAMA3 = dict(base=500000.0, factor=8.0, low_freq_factor=1.0, high_freq_factor=4.0, original_max_position=8192)
YARN = dict(base=10000.0, factor=40.0, beta_fast=32.0, beta_slow=1.0, original_max_position=4096)
LINEAR = dict(base=10000.0, factor=4.0)
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token of a 32/8-head model: what a single-user decode step pays per layer
        dict(name="rope one token", op="rope", tokens=1, hq=32, hk=8, d=128, rot=128, inter=False, scaling="llama3",
             far=131072, strided=False),
        # a whole prompt through the same layer, q and k sliced out of the fused projection
        dict(name="rope prompt", op="rope", tokens=8191, hq=32, hk=8, d=128, rot=128, inter=False, scaling="llama3",
             far=131072, strided=True),
        # latent attention's 64 rope dims of 128 heads (interleaved pairs, 128 other dims between them)
        dict(name="rope latent q", op="rope", tokens=2048, hq=128, hk=1, d=64, rot=64, inter=True, scaling="yarn",
             far=163840, strided=True),
        # a decode step of 128 sequences at long contexts: one row each, every row in another page
        dict(name="append 128 decodes", op="append", lens=1, nd=128, nc=0, cl=0, ctx=131072, hq=32, hkv=8, d=128,
             rot=128, inter=False, scaling="llama3", ps=16, kv="bf16", pad=0, strided=True),
        # decodes beside two prompt chunks into an fp8 cache with scales, half of the head rotated
        dict(name="append mixed fp8", op="append", lens=2, nd=61, nc=2, cl=1021, ctx=8192, hq=16, hkv=8, d=256,
             rot=128, inter=False, scaling="linear", ps=32, kv="fp8", pad=5, strided=False),
        # long prompts filling a bf16 cache
        dict(name="append prompts", op="append", lens=3, nd=0, nc=4, cl=4096, ctx=32768, hq=32, hkv=8, d=128, rot=128,
             inter=False, scaling="llama3", ps=16, kv="bf16", pad=0, strided=True),
        # a decoder's next token over a short encoder input, a handful of sequences
        dict(name="cross few decodes", op="cross", lens=4, n=4, q0=1, q1=1, s0=40, s1=300, empty=0, hq=16, hkv=16, d=64,
             ps=16, kv="bf16", pad=0),
        # a full decode batch over encoder states of about 1500 positions, multi-head
        dict(name="cross 64 decodes", op="cross", lens=5, n=64, q0=1, q1=1, s0=1400, s1=1500, empty=1, hq=20, hkv=20,
             d=64, ps=64, kv="bf16", pad=0),
        # decoder prompts of uneven length over the same encoder states
        dict(name="cross prompts", op="cross", lens=6, n=16, q0=4, q1=448, s0=700, s1=1500, empty=1, hq=20, hkv=20, d=64,
             ps=64, kv="bf16", pad=7),
        # long documents on both sides, grouped heads
        dict(name="cross long", op="cross", lens=7, n=4, q0=4096, q1=4096, s0=4096, s1=4096, empty=0, hq=32, hkv=8, d=128,
             ps=16, kv="bf16", pad=0),
        # a serving step: 128 decodes and 2 prompt chunks, rotated, written and attended
        dict(name="step mixed", op="step", lens=8, nd=128, nc=2, cl=512, c0=512, ctx=4096, hq=32, hkv=8, d=128, rot=128,
             inter=False, scaling="llama3", ps=16, kv="bf16", pad=0, strided=True),
        # a small decode batch over an fp8 cache
        dict(name="step few decodes fp8", op="step", lens=9, nd=7, nc=0, cl=0, c0=100, ctx=3000, hq=16, hkv=8, d=128,
             rot=64, inter=True, scaling="none", ps=32, kv="fp8", pad=1, strided=False),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["rope", "append", "cross", "step"])
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 6, 8])
    c = dict(op=op, lens=rng.randrange(1 << 20))
    rot = dict(rot=rng.choice([d, d, d // 2, 32]), inter=rng.random() < 0.4,
               scaling=rng.choice(["none", "linear", "llama3", "yarn"]), strided=rng.random() < 0.5)
    kv = rng.choice(["bf16", "bf16", "fp8"])
    ps = rng.choice([8, 16, 32, 64])
    if op == "rope":
        c.update(tokens=_log(rng, 1, 8000), hq=hkv * g, hk=hkv, d=d, far=_log(rng, 100, 1000000), **rot)
    elif op == "append":
        nc = rng.choice([0, 1, 3])
        c.update(nd=_log(rng, 1, 200), nc=nc, cl=_log(rng, 17, 2500) if nc else 0, ctx=_log(rng, 3000, 100000), hq=hkv * g,
                 hkv=hkv, d=d, ps=ps, kv=kv, pad=rng.choice([0, 3]), **rot)
    elif op == "cross":
        n, q1, s1 = _log(rng, 1, 48), _log(rng, 1, 900), _log(rng, 30, 4000)
        n = max(1, min(n, int(4e11 / (4 * q1 * s1 * hkv * g * d))))
        c.update(n=n, q0=rng.choice([1, q1]), q1=q1, s0=rng.randint(1, s1), s1=s1, empty=rng.choice([0, 1]) if n > 1 else 0,
                 hq=hkv * g, hkv=hkv, d=d, ps=ps, kv=kv, pad=rng.choice([0, 3]))
    else:
        nc = rng.choice([0, 1, 2])
        c.update(nd=_log(rng, 1, 100), nc=nc, cl=_log(rng, 17, 500) if nc else 0, c0=500, ctx=_log(rng, 600, 4000),
                 hq=hkv * g, hkv=hkv, d=d, ps=ps, kv=kv, pad=rng.choice([0, 3]), **rot)
    return c


def _lens(c):
    """(query lengths, key lengths) of a case's sequences: part of the case, the same for every seed."""
    r = random.Random(c["lens"])
    if c["op"] == "cross":
        ql = [r.randint(c["q0"], c["q1"]) for _ in range(c["n"])]
        kl = [r.randint(c["s0"], c["s1"]) for _ in range(c["n"])]
        for i in range(c["empty"]):
            kl[(7 * i + 1) % c["n"]] = 0
        return ql, kl
    ql = [1] * c["nd"] + [c["cl"]] * c["nc"]
    low = c.get("c0", 1)
    return ql, [r.randint(max(low, n), max(low, n, c["ctx"])) for n in ql]


def _esz(c):
    return 1 if c["kv"] == "fp8" else 2


def work(c):
    d, hq = c["d"], c["hq"]
    if c["op"] == "rope":
        n = c["tokens"] * (hq + c["hk"])
        return {"bytes": 4 * n * d, "flops": 3 * n * c["rot"]}
    ql, kl = _lens(c)
    t, hkv = sum(ql), c["hkv"]
    row = 2 * hkv * d * _esz(c)  # one token's K and V in the cache
    if c["op"] == "append":
        return {"bytes": 4 * t * hq * d + 2 * t * 2 * hkv * d + t * row, "flops": 3 * t * (hq + hkv) * c["rot"]}
    if c["op"] == "cross":
        return {"bytes": 4 * t * hq * d + sum(k for q, k in zip(ql, kl) if q) * row,
                "flops": 4 * d * hq * sum(q * k for q, k in zip(ql, kl))}
    # a query sees the keys up to its own: k - (q - 1) / 2 on average over a chunk's last q of k keys
    return {"bytes": 4 * t * hq * d + 2 * t * 2 * hkv * d + sum(kl) * row,
            "flops": 4 * d * hq * sum(q * (k - (q - 1) / 2) for q, k in zip(ql, kl))}


# ------------------------------------------------------------------ inputs
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def _qkv(g, t, hq, hk, hv, d, strided):
    """q, k, v [t, heads, d]: slices of one projection's output, or tensors of their own."""
    if not strided:
        return tuple(_randn(g, t, h, d) if h else None for h in (hq, hk, hv))
    x = _randn(g, t, (hq + hk + hv) * d)
    cut = [x[:, a * d:(a + h) * d].unflatten(1, (h, d)) if h else None for a, h in ((0, hq), (hq, hk), (hq + hk, hv))]
    return tuple(cut)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, s = case, {"case": case, "table": None}
    if c["op"] != "cross":
        s["frequencies"] = _frequencies(c)
    if c["op"] == "rope":
        t, d = c["tokens"], c["d"]
        if c["d"] == 64 and c["strided"]:  # the last 64 of each head's 192 dims
            s["q"] = _randn(g, t, c["hq"], 192)[..., 128:]
            s["k"] = _randn(g, t, c["hk"], d)
        else:
            s["q"], s["k"], _ = _qkv(g, t, c["hq"], c["hk"], 0, d, c["strided"])
        s["positions"] = torch.randint(0, c["far"], (t,), generator=g, device="cuda", dtype=torch.int32)
        s["q_out"] = torch.zeros(t, c["hq"], d, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.zeros(t, c["hk"], d, dtype=torch.bfloat16, device="cuda")
        return s
    ql, kl = _lens(c)
    n, t, ps, hq, hkv, d = len(ql), sum(ql), c["ps"], c["hq"], c["hkv"], c["d"]
    slots = n + 2  # two sequence slots of the batch's tables are unused
    pps = max(1, -(-max(kl) // ps))
    # pages the call touches: those of the new rows (append), every page of a sequence (cross, step)
    first = [(k - q) // ps if c["op"] == "append" else 0 for q, k in zip(ql, kl)]
    count = [-(-k // ps) - f for f, k in zip(first, kl)]
    total = sum(count) + 3
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.randint(0, total, (slots, pps), generator=g, device="cuda", dtype=torch.int32)
    at = np.concatenate([np.arange(f, f + m) + i * pps for i, (f, m) in enumerate(zip(first, count))])
    table.view(-1)[torch.from_numpy(at).cuda()] = perm[:sum(count)]
    kv = _randn(g, total * ps, 2 * hkv, d).view(total, ps, 2 * hkv, d)
    s["kv"] = kv.to(E4M3) if c["kv"] == "fp8" else kv
    s["scales"] = (0.03125, 0.0625) if c["kv"] == "fp8" and c["op"] != "cross" else (0.5, 2.0) if c["kv"] == "fp8" else (None, None)
    s["page_indices"] = table
    s["kv_lens"] = torch.tensor(kl + [0] * (slots - n), dtype=torch.int32, device="cuda")
    s["cu_q_lens"] = torch.tensor(np.concatenate([[0], np.cumsum(ql), [t] * (slots - n)]), dtype=torch.int32, device="cuda")
    s["num_seqs"] = torch.tensor([n], dtype=torch.int32, device="cuda")
    s["n"], s["t"], s["sm_scale"] = n, t, d ** -0.5
    rows = t + c["pad"]
    if c["op"] == "cross":
        s["q"] = _randn(g, rows, hq, d)
    else:
        s["q"], s["k"], s["v"] = _qkv(g, rows, hq, hkv, hkv, d, c["strided"])
        s["q_out"] = torch.zeros(rows, hq, d, dtype=torch.bfloat16, device="cuda")
    s["out"] = torch.zeros(rows, hq, d, dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------ the calls
def _table(s):
    """The rotation's table, as a program makes it once from its configuration and keeps it."""
    if s["table"] is None:
        from ragged_paged_attention_gb300 import api
        c = s["case"]
        more = {"llama3": LLAMA3, "yarn": YARN, "linear": LINEAR, "none": dict(base=10000.0)}[c["scaling"]]
        scaling = dict(type=c["scaling"], **{k: v for k, v in more.items() if k != "base"})
        s["table"] = api.make_rope_table(c["rot"], base=more["base"], interleaved=c["inter"],
                                         scaling=None if c["scaling"] == "none" else scaling)
    return s["table"]


def _own(s):
    from ragged_paged_attention_gb300 import api
    c = s["case"]
    if c["op"] == "rope":
        q, k = api.rope_apply(s["q"], s["k"], s["positions"], _table(s), q_out=s["q_out"], k_out=s["k_out"])
        return {"q": q, "k": k}
    batch = (s["kv"], s["kv_lens"], s["page_indices"], s["cu_q_lens"], s["num_seqs"])
    ks, vs = s["scales"]
    if c["op"] == "append":
        q, kv = api.rpa_rope_update_kv_cache(s["q"], s["k"], s["v"], *batch, _table(s), k_scale=ks, v_scale=vs,
                                             q_out=s["q_out"])
        return {"q": q, "kv": kv}
    if c["op"] == "cross":
        return {"out": api.rpa_cross_forward(s["q"], *batch, sm_scale=s["sm_scale"], k_scale=ks, v_scale=vs, out=s["out"])}
    out = api.rpa_rope_forward_update(s["q"], s["k"], s["v"], *batch, _table(s), sm_scale=s["sm_scale"], k_scale=ks,
                                      v_scale=vs, q_rot=s["q_out"], out=s["out"])
    return {"out": out, "kv": s["kv"]}


# ------------------------------------------------------------------ plain forms
def _frequencies(c):
    """(angle per position of each pair, amplitude), float64."""
    r, kind = c["rot"], c["scaling"]
    p = {"llama3": LLAMA3, "yarn": YARN, "linear": LINEAR, "none": dict(base=10000.0)}[kind]
    i = torch.arange(0, r, 2, dtype=torch.float64, device="cuda")
    f = p["base"] ** (-i / r)
    if kind == "linear":
        return f / p["factor"], 1.0
    if kind == "llama3":
        turns = p["original_max_position"] * f / (2 * math.pi)
        keep = ((turns - p["low_freq_factor"]) / (p["high_freq_factor"] - p["low_freq_factor"])).clamp(0, 1)
        return keep * f + (1 - keep) * f / p["factor"], 1.0
    if kind == "yarn":
        def dim(turns):
            return r * math.log(p["original_max_position"] / (turns * 2 * math.pi)) / (2 * math.log(p["base"]))
        low, high = max(math.floor(dim(p["beta_fast"])), 0), min(math.ceil(dim(p["beta_slow"])), r - 1)
        ramp = ((i / 2 - low) / max(high - low, 0.001)).clamp(0, 1)
        return ramp * f / p["factor"] + (1 - ramp) * f, 0.1 * math.log(p["factor"]) + 1
    return f, 1.0


def _rotate(s, x, pos):
    """x [t, heads, d] float32, rotated to the positions pos [t]."""
    c, (f, amp) = s["case"], s["frequencies"]
    angle = pos.double()[:, None, None] * f
    cos, sin = (amp * angle.cos()).float(), (amp * angle.sin()).float()
    r = c["rot"]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["inter"] else (x[..., :r // 2], x[..., r // 2:r])
    y, z = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([y, z], -1).flatten(-2) if c["inter"] else torch.cat([y, z], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _tokens(s):
    """Each token's sequence, place in it and position."""
    tok = torch.arange(s["t"], device="cuda")
    cu, n = s["cu_q_lens"].long(), s["n"]
    seq = torch.searchsorted(cu[1:n + 1].contiguous(), tok, right=True)
    j = tok - cu[seq]
    return seq, j, s["kv_lens"].long()[seq] - (cu[seq + 1] - cu[seq]) + j


def _store(x, scale, like):
    """x float32 as the cache holds it."""
    x = x if scale is None else x / scale
    return x.clamp(-448, 448).to(E4M3).view(torch.uint8) if like.dtype == E4M3 else x.to(torch.bfloat16)


def _append(s):
    """Writes q_out and the cache; returns each token's sequence and place in it."""
    c, t, kv = s["case"], s["t"], s["kv"]
    seq, j, pos = _tokens(s)
    ps = c["ps"]
    slot = s["page_indices"][seq, pos // ps].long() * ps + pos % ps
    s["q_out"][:t] = _rotate(s, s["q"][:t].float(), pos).to(torch.bfloat16)
    flat = (kv.view(torch.uint8) if kv.dtype == E4M3 else kv).view(-1, 2 * c["hkv"], c["d"])
    flat[slot, 0::2] = _store(_rotate(s, s["k"][:t].float(), pos), s["scales"][0], kv)
    flat[slot, 1::2] = _store(s["v"][:t].float(), s["scales"][1], kv)
    return seq, j


def _attend(s, q, lo, hi, qm, causal):
    """Attention of sequences lo..hi (at most qm queries each) over their cached keys: [hi - lo, qm, hq, d] float32."""
    c, kv = s["case"], s["kv"]
    ps, hkv, d, hq = c["ps"], c["hkv"], c["d"], c["hq"]
    lens, cu = s["kv_lens"][lo:hi].long(), s["cu_q_lens"].long()
    most = s["page_indices"].shape[1] * ps
    key = torch.arange(most, device="cuda")
    slot = (s["page_indices"][lo:hi].long()[:, :, None] * ps + torch.arange(ps, device="cuda")).flatten(1)
    flat = (kv.view(torch.uint8) if kv.dtype == E4M3 else kv).view(-1, 2 * hkv, d)
    x = flat[slot]
    x = x.view(E4M3).float() if kv.dtype == E4M3 else x.float()
    k, v = x[:, :, 0::2], x[:, :, 1::2]
    if s["scales"][0] is not None:
        k, v = (k * s["scales"][0]).bfloat16().float(), (v * s["scales"][1]).bfloat16().float()
    tok = cu[lo:hi, None] + torch.arange(qm, device="cuda")
    q = q[tok.clamp(max=q.shape[0] - 1)].float()  # [m, qm, hq, d]
    m, g = hi - lo, hq // hkv
    q = q.view(m, qm, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(m, hkv, g * qm, d)
    score = (q @ k.permute(0, 2, 3, 1)) * s["sm_scale"]
    last = lens[:, None] - 1
    if causal:
        last = last - (cu[lo + 1:hi + 1] - cu[lo:hi])[:, None] + 1 + torch.arange(qm, device="cuda")
        last = last.repeat(1, g)
    score.masked_fill_((key > last[..., None])[:, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (score - top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ v.permute(0, 2, 1, 3)) / total.masked_fill(total == 0, 1.0)
    return o.view(m, hkv, g, qm, d).permute(0, 3, 1, 2, 4).reshape(m, qm, hq, d)


def _plain(s):
    c = s["case"]
    if c["op"] == "rope":
        for x in "qk":
            s[x + "_out"].copy_(_rotate(s, s[x].float(), s["positions"]))
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["op"] == "append":
        _append(s)
        return {"q": s["q_out"], "kv": s["kv"]}
    if c["op"] == "cross":
        seq, j, _ = _tokens(s)
        s["out"][:s["t"]] = _attend(s, s["q"], 0, s["n"], max(_lens(c)[0]), False)[seq, j].to(torch.bfloat16)
        return {"out": s["out"]}
    seq, j = _append(s)
    nd = c["nd"]
    s["out"][:nd] = _attend(s, s["q_out"], 0, nd, 1, True)[:, 0].to(torch.bfloat16)
    if c["nc"]:
        s["out"][nd:s["t"]] = _attend(s, s["q_out"], nd, s["n"], c["cl"], True).flatten(0, 1).to(torch.bfloat16)
    return {"out": s["out"], "kv": s["kv"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits
def _turned(c, x, positions):
    """float64 [t, heads, d] rotated: each pair as a complex number times A e^(i p f)."""
    r, kind, f, amp = c["rot"], c["scaling"], [], 1.0
    for i in range(r // 2):
        w = {"llama3": 500000.0}.get(kind, 10000.0) ** (-2.0 * i / r)
        if kind == "linear":
            w /= 4.0
        elif kind == "llama3":
            wave = 2.0 * math.pi / w
            if wave > 8192.0 / 1.0:
                w /= 8.0
            elif wave >= 8192.0 / 4.0:
                smooth = (8192.0 / wave - 1.0) / 3.0
                w = (1.0 - smooth) * w / 8.0 + smooth * w
        elif kind == "yarn":
            def edge(turns):
                return r * math.log(4096.0 / (2.0 * math.pi * turns)) / math.log(10000.0) / 2.0
            a, b = max(0, math.floor(edge(32.0))), min(r - 1, math.ceil(edge(1.0)))
            mix = min(1.0, max(0.0, (i - a) / (b - a if b > a else 0.001)))
            w = w * (1.0 - mix) + w / 40.0 * mix
            amp = 1.0 + 0.1 * math.log(40.0)
        f.append(w)
    phase = positions.double()[:, None] * torch.tensor(f, dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.full_like(phase, amp), phase)[:, None, :]
    y = x.clone()
    if c["inter"]:
        y[..., :r] = torch.view_as_real(torch.view_as_complex(x[..., :r].unflatten(-1, (r // 2, 2)).contiguous()) * turn).flatten(-2)
    else:
        z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * turn
        y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
    return y


def _held(x, scale, fp8):
    """float64 values of x in the cache's type (round to nearest even, e4m3 saturating)."""
    if not fp8:
        return x.to(torch.bfloat16).double()
    x = x / scale
    exponent = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))).clamp(min=-6.0)
    unit = torch.exp2(exponent - 3.0)
    return (torch.round(x / unit) * unit).clamp(-448.0, 448.0)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        return {x: _turned(c, s[x].double(), s["positions"]) for x in "qk"}
    ql, kl = _lens(c)
    ps, hkv, d, g, fp8 = c["ps"], c["hkv"], c["d"], c["hq"] // c["hkv"], c["kv"] == "fp8"
    cache = s["kv"].double().view(-1, 2 * hkv, d)
    pages = s["page_indices"].cpu().long()
    rows = s["q"].shape[0]
    q, out = s["q"].double(), torch.zeros(rows, c["hq"], d, dtype=torch.float64, device="cuda")
    place = [(pages[i, :, None] * ps + torch.arange(ps)).flatten()[:k] for i, k in enumerate(kl)]  # each key's row
    starts = np.concatenate([[0], np.cumsum(ql)]).tolist()
    if c["op"] != "cross":
        position = torch.cat([torch.arange(k - n, k) for n, k in zip(ql, kl)]).cuda()
        row = torch.cat([p[k - n:] for p, n, k in zip(place, ql, kl)]).cuda()
        t = starts[-1]
        cache[row, 0::2] = _held(_turned(c, s["k"][:t].double(), position), s["scales"][0], fp8)
        cache[row, 1::2] = _held(s["v"][:t].double(), s["scales"][1], fp8)
        q = _turned(c, q[:t], position)
        if c["op"] == "append":
            out[:t] = q
            return {"q": out, "kv": cache.view(s["kv"].shape)}
        q = q.to(torch.bfloat16).double()  # attention takes the rotated queries in bf16
    for i, (n, k) in enumerate(zip(ql, kl)):
        if n == 0 or k == 0:
            continue
        a = starts[i]
        x = cache[place[i].cuda()]
        keys, values = x[:, 0::2], x[:, 1::2]
        if s["scales"][0] is not None:
            keys, values = ((y.float() * z).bfloat16().double() for y, z in zip((keys, values), s["scales"]))
        for h in range(hkv):
            w = torch.einsum("qgd,kd->gqk", q[a:a + n, h * g:(h + 1) * g], keys[:, h]) * s["sm_scale"]
            if c["op"] == "step":
                future = torch.arange(k, device="cuda")[None, :] > torch.arange(k - n, k, device="cuda")[:, None]
                w.masked_fill_(future, -math.inf)
            out[a:a + n, h * g:(h + 1) * g] = torch.einsum("gqk,kd->qgd", torch.softmax(w, -1), values[:, h])
    if c["op"] == "cross":
        return {"out": out}
    return {"out": out, "kv": cache.view(s["kv"].shape)}
