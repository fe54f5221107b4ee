"""Cases of the operators that keep long contexts in less memory, with their plain forms.

``store``    new K/V rows, turned, to pages that hold them in 4 bits with a scale and a minimum a
             group (``api.rpa_g4_update_kv_cache``), then read back (``api.rpa_g4_read_kv_cache``)
``attend``   causal attention over such pages (``api.rpa_g4_forward``)
``weights``  what each cached key gets of the batch's attention, summed over the queries that share
             its head and added to what it had before (``api.rpa_key_weights``)
``evict``    the keys of the largest weights kept, and moved to the front of their sequence's pages
             (``api.rpa_evict_kv_cache``)

With ``own`` false ``run`` computes them from elementary torch operations in float32 (rotations in
float64); ``exact`` restates them in float64.

A 4-bit row: of a group of 64 values (32 where head_dim is 64), as bf16 holds them, m is the least and
s the bf16 nearest to (greatest - least) / 15; x is held as n = round((x - m) / s) in 0..15, and read
as s n + m.  A token's K and V of one head lie in one row: K's values, two a byte (the even one in
the low half), V's, then s and m of K's groups and of V's, then unused bytes up to a multiple of 16.
"""
import math
import random

import numpy as np
import torch

own = False

LLAMA3 = dict(base=500000.0, factor=8.0, low_freq_factor=1.0, high_freq_factor=4.0, original_max_position=8192)
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step of 64 sequences at long contexts: a row each, every row in another page
        dict(name="store 64 decodes", op="store", lens=1, nd=64, nc=0, cl=0, c0=1, ctx=100000, hq=32, hkv=8, d=128, rot=128,
             inter=False, scaling="llama3", ps=16, pad=0, strided=True),
        # decodes beside two prompt chunks of wide heads, half of the head turned, rows of padding behind
        dict(name="store mixed", op="store", lens=2, nd=61, nc=2, cl=1021, c0=1, ctx=8192, hq=16, hkv=8, d=256, rot=128,
             inter=True, scaling="none", ps=32, pad=5, strided=False),
        # long prompts filling the cache
        dict(name="store prompts", op="store", lens=3, nd=0, nc=4, cl=4096, c0=1, ctx=32768, hq=32, hkv=8, d=128, rot=128,
             inter=False, scaling="llama3", ps=16, pad=0, strided=True),
        # the next token of a handful of sequences: latency counts
        dict(name="attend few decodes", op="attend", lens=4, nd=5, nc=0, cl=0, c0=100, ctx=3000, hq=16, hkv=8, d=128, ps=16,
             window=0, cap=0.0, pad=0),
        # a full decode batch over contexts of up to 8192
        dict(name="attend 128 decodes", op="attend", lens=5, nd=128, nc=0, cl=0, c0=512, ctx=8192, hq=32, hkv=8, d=128, ps=16,
             window=0, cap=0.0, pad=0),
        # decodes and prompt chunks of wide heads with a window and a soft cap
        dict(name="attend mixed", op="attend", lens=6, nd=64, nc=2, cl=1024, c0=1024, ctx=8192, hq=16, hkv=8, d=256, ps=32,
             window=4096, cap=50.0, pad=3),
        # whole prompts
        dict(name="attend prompts", op="attend", lens=7, nd=0, nc=4, cl=4096, c0=4096, ctx=4096, hq=32, hkv=8, d=128, ps=16,
             window=0, cap=0.0, pad=0),
        # the weights that a decode step of 96 sequences gives the keys of a bf16 cache
        dict(name="weights 96 decodes", op="weights", lens=8, nd=96, nc=0, cl=0, c0=2000, ctx=8192, hq=32, hkv=8, d=128,
             ps=16, kv="bf16", keep=1.0, window=0, cap=0.0),
        # a few long sequences in a 4-bit cache, earlier weights fading
        dict(name="weights few decodes g4", op="weights", lens=9, nd=6, nc=0, cl=0, c0=100, ctx=20000, hq=16, hkv=8, d=128,
             ps=16, kv="g4", keep=0.9, window=0, cap=0.0),
        # the last 32 queries of long prompts vote on which of its keys stay
        dict(name="weights windows", op="weights", lens=10, nd=0, nc=8, cl=32, c0=8000, ctx=16000, hq=32, hkv=8, d=128, ps=16,
             kv="bf16", keep=0.0, window=0, cap=0.0),
        # one sequence that has grown past its budget
        dict(name="evict one", op="evict", lens=11, n=1, c0=3001, ctx=3001, keep=1024, sinks=4, recent=128, hkv=8, d=128, ps=16,
             kv="bf16"),
        # a batch cut back to 2048 keys a head
        dict(name="evict batch", op="evict", lens=12, n=48, c0=4000, ctx=12000, keep=2048, sinks=4, recent=256, hkv=8, d=128,
             ps=16, kv="bf16"),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["store", "attend", "weights", "evict"])
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 6, 8])
    ps = rng.choice([8, 16, 32, 64])
    c = dict(op=op, lens=rng.randrange(1 << 20), hkv=hkv, d=d, ps=ps)
    if op == "evict":
        ctx = _log(rng, 20, 20000)
        c.update(n=_log(rng, 1, 40), c0=rng.randint(1, ctx), ctx=ctx, keep=max(1, int(ctx * rng.uniform(0.1, 0.9))),
                 sinks=rng.choice([0, 1, 4]), recent=rng.choice([0, 13, 64]), kv=rng.choice(["bf16", "fp8"]))
        c["n"] = max(1, min(c["n"], 300000 // ctx))
        return c
    nc = rng.choice([0, 1, 3])
    c.update(nd=_log(rng, 1, 100), nc=nc, hq=hq)
    if op == "store":
        c.update(cl=_log(rng, 17, 2500) if nc else 0, c0=1, ctx=_log(rng, 3000, 100000), rot=rng.choice([d, d, d // 2, 32]),
                 inter=rng.random() < 0.4, scaling=rng.choice(["none", "llama3"]), strided=rng.random() < 0.5,
                 pad=rng.choice([0, 3]))
        return c
    c.update(cl=_log(rng, 3, 1000) if nc else 0, c0=rng.choice([1, 500]), ctx=_log(rng, 600, 8000),
             window=rng.choice([0, 0, 0, rng.randint(1, 3000)]), cap=rng.choice([0.0, 0.0, 30.0]))
    if op == "attend":
        c.update(pad=rng.choice([0, 3]))
    else:
        c.update(kv=rng.choice(["bf16", "g4"]), keep=rng.choice([0.0, 0.75, 1.0]))
    return c


def _lens(c):
    """(query lengths, key lengths) of a case's sequences: part of the case, the same for every seed."""
    r = random.Random(c["lens"])
    ql = [1] * c["n"] if c["op"] == "evict" else [1] * c["nd"] + [c["cl"]] * c["nc"]
    low = c["c0"]
    return ql, [r.randint(max(low, n), max(low, n, c["ctx"])) for n in ql]


def _group(d):
    return 32 if d == 64 else 64


def _row_bytes(d):
    return (d + 8 * (d // _group(d)) + 15) // 16 * 16


def _seen(c, q, k):
    """(query, key) pairs of a sequence, and the keys that any of its queries sees."""
    if not c["window"]:
        return q * (k - (q - 1) / 2), k
    w = c["window"]
    pairs = sum(min(w, k - q + 1 + i) for i in range(q))
    return pairs, min(k, q - 1 + w)


def work(c):
    d, hkv = c["d"], c["hkv"]
    ql, kl = _lens(c)
    t = sum(ql)
    if c["op"] == "evict":
        # the weights read, the kept ones and the places that keys came from written; of the kept keys a share
        # of about 1 - keep / length lies behind and moves
        row = 2 * d * (1 if c["kv"] == "fp8" else 2)
        kept = [min(k, max(c["keep"], c["sinks"] + c["recent"])) for k in kl]
        moved = sum(n * (1 - n / k) for n, k in zip(kept, kl))
        return {"bytes": hkv * (4 * sum(kl) + 8 * sum(kept) + 2 * row * moved), "flops": hkv * sum(kl)}
    hq = c["hq"]
    if c["op"] == "store":
        held = d + 8 * (d // _group(d))
        # q read and written, k and v read, written as held, read as held and written as bf16
        return {"bytes": 4 * t * hq * d + 2 * t * hkv * (2 * d + held + 2 * d), "flops": 3 * t * (hq + hkv) * c["rot"] + 12 * t * hkv * d}
    seen = [_seen(c, q, k) for q, k in zip(ql, kl)]
    if c["op"] == "attend":
        return {"bytes": 4 * t * hq * d + sum(k for _, k in seen) * hkv * (d + 8 * (d // _group(d))),
                "flops": 4 * d * hq * sum(p for p, _ in seen)}
    row = 2 * d if c["kv"] == "bf16" else (d + 8 * (d // _group(d))) / 2
    return {"bytes": 2 * t * hq * d + hkv * (sum(k for _, k in seen) * row + sum(kl) * 8), "flops": 2 * d * hq * sum(p for p, _ in seen)}


# ------------------------------------------------------------------ inputs
def _randn(g, *shape):
    """bf16 normal values, none beyond two deviations: a row after its normalisation."""
    return torch.randn(*shape, generator=g, device="cuda").clamp_(-2, 2).to(torch.bfloat16)


def _qkv(g, t, hq, hkv, d, strided):
    """q, k, v [t, heads, d]: slices of one projection's output, or tensors of their own."""
    if not strided:
        return tuple(_randn(g, t, h, d) for h in (hq, hkv, hkv))
    x = _randn(g, t, (hq + 2 * hkv) * d)
    return tuple(x[:, a * d:(a + h) * d].unflatten(1, (h, d)) for a, h in ((0, hq), (hq, hkv), (hq + hkv, hkv)))


def _g4_pages(g, slots, hkv, d):
    """Pages of 4-bit rows as a run of writes leaves them: any values, scales about 0.3, minima about -2.4."""
    n = d // _group(d)
    pages = torch.randint(0, 256, (slots, hkv, _row_bytes(d)), generator=g, device="cuda", dtype=torch.uint8)
    u = torch.rand(slots, hkv, 2 * n, 2, generator=g, device="cuda")
    sm = torch.stack([0.22 + 0.16 * u[..., 0], -2.9 + u[..., 1]], -1).to(torch.bfloat16)
    pages[..., d:d + 8 * n] = sm.flatten(2).view(torch.uint8)
    return pages


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, s = case, {"case": case, "table": None}
    ql, kl = _lens(c)
    n, t, ps, hkv, d = len(ql), sum(ql), c["ps"], c["hkv"], c["d"]
    slots = n + 2  # two sequence slots of the batch's tables are unused
    pps = max(1, -(-max(kl) // ps))
    # pages the call touches: those of the new rows (store), else every page of a sequence
    first = [(k - q) // ps if c["op"] == "store" else 0 for q, k in zip(ql, kl)]
    count = [-(-k // ps) - f for f, k in zip(first, kl)]
    total = sum(count) + 3
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.randint(0, total, (slots, pps), generator=g, device="cuda", dtype=torch.int32)
    at = np.concatenate([np.arange(f, f + m) + i * pps for i, (f, m) in enumerate(zip(first, count))])
    table.view(-1)[torch.from_numpy(at).cuda()] = perm[:sum(count)]
    s["page_indices"] = table
    s["kv_lens"] = torch.tensor(kl + [0] * (slots - n), dtype=torch.int32, device="cuda")
    s["cu_q_lens"] = torch.tensor(np.concatenate([[0], np.cumsum(ql), [t] * (slots - n)]), dtype=torch.int32, device="cuda")
    s["num_seqs"] = torch.tensor([n], dtype=torch.int32, device="cuda")
    s["n"], s["t"], s["sm_scale"], s["most"] = n, t, d ** -0.5, pps * ps
    if c["op"] in ("store", "attend") or c.get("kv") == "g4":
        s["kv"] = _g4_pages(g, total * ps, hkv, d).view(total, ps, hkv, _row_bytes(d))
    else:
        kv = _randn(g, total * ps, 2 * hkv, d).view(total, ps, 2 * hkv, d)
        s["kv"] = kv.to(E4M3) if c["kv"] == "fp8" else kv
    rows = t + c.get("pad", 0)
    if c["op"] == "store":
        s["frequencies"] = _frequencies(c)
        s["q"], s["k"], s["v"] = _qkv(g, rows, c["hq"], hkv, d, c["strided"])
        s["q_out"] = torch.zeros(rows, c["hq"], d, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.zeros(rows, hkv, d, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.zeros(rows, hkv, d, dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "evict":
        # few keys carry most of the weight
        s["weights"] = torch.rand(total, hkv, ps, generator=g, device="cuda").pow_(6)
        s["weights_out"] = torch.zeros_like(s["weights"])
        s["budgets"] = torch.tensor([c["keep"]] * slots, dtype=torch.int32, device="cuda")
        s["kept"] = max(c["keep"], c["sinks"] + c["recent"])
        s["lens_out"] = torch.zeros(slots, dtype=torch.int32, device="cuda")
        s["slots_out"] = torch.zeros(slots, hkv, s["kept"], dtype=torch.int32, device="cuda")
    else:
        s["q"] = _randn(g, rows, c["hq"], d)
        if c["op"] == "attend":
            s["out"] = torch.zeros(rows, c["hq"], d, dtype=torch.bfloat16, device="cuda")
        else:
            s["weights"] = torch.rand(total, hkv, ps, generator=g, device="cuda").pow_(6)
            s["weights_out"] = torch.zeros_like(s["weights"])
    return s


# ------------------------------------------------------------------ the calls
def _table(s):
    """The rotation's table, as a program makes it once from its configuration and keeps it."""
    if s["table"] is None:
        from ragged_paged_attention_gb300 import api
        c = s["case"]
        scaling = dict(type="llama3", **{k: v for k, v in LLAMA3.items() if k != "base"})
        s["table"] = (api.make_rope_table(c["rot"], base=500000.0, interleaved=c["inter"], scaling=scaling)
                      if c["scaling"] == "llama3" else api.make_rope_table(c["rot"], base=10000.0, interleaved=c["inter"]))
    return s["table"]


def _own(s):
    from ragged_paged_attention_gb300 import api
    c = s["case"]
    if c["op"] == "evict":
        lens, places = api.rpa_evict_kv_cache(s["kv"], s["kv_lens"], s["page_indices"], s["num_seqs"], s["weights"], s["budgets"],
                                              s["kept"], sinks=c["sinks"], recent=c["recent"], kv_lens_out=s["lens_out"],
                                              slots_out=s["slots_out"], weights_out=s["weights_out"])
        return {"lens": lens, "slots": places, "weights": s["weights_out"], "kv": s["kv"]}
    batch = (s["kv"], s["kv_lens"], s["page_indices"], s["cu_q_lens"], s["num_seqs"])
    if c["op"] == "store":
        q, _ = api.rpa_g4_update_kv_cache(s["q"], s["k"], s["v"], *batch, _table(s), q_out=s["q_out"])
        k, v = api.rpa_g4_read_kv_cache(*batch, k_out=s["k_out"], v_out=s["v_out"])
        return {"q": q, "k": k, "v": v}
    window, cap = c["window"] or None, c["cap"] or None
    if c["op"] == "attend":
        return {"out": api.rpa_g4_forward(s["q"], *batch, sm_scale=s["sm_scale"], sliding_window=window, soft_cap=cap, out=s["out"])}
    return {"weights": api.rpa_key_weights(s["q"], *batch, s["weights"], sm_scale=s["sm_scale"], sliding_window=window,
                                           soft_cap=cap, keep=c["keep"], weights_out=s["weights_out"])}


# ------------------------------------------------------------------ plain forms
def _frequencies(c):
    """Angle per position of each pair, float64."""
    r, p = c["rot"], LLAMA3
    i = torch.arange(0, r, 2, dtype=torch.float64, device="cuda")
    if c["scaling"] == "none":
        return 10000.0 ** (-i / r)
    f = p["base"] ** (-i / r)
    turns = p["original_max_position"] * f / (2 * math.pi)
    keep = ((turns - p["low_freq_factor"]) / (p["high_freq_factor"] - p["low_freq_factor"])).clamp(0, 1)
    return keep * f + (1 - keep) * f / p["factor"]


def _rotate(s, x, pos):
    """x [t, heads, d] bf16 turned to the positions pos [t], in bf16: in float64, since what lies at a step's border counts."""
    c, x = s["case"], x.double()
    angle = pos.double()[:, None, None] * s["frequencies"]
    cos, sin = angle.cos(), angle.sin()
    r = c["rot"]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["inter"] else (x[..., :r // 2], x[..., r // 2:r])
    y, z = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([y, z], -1).flatten(-2) if c["inter"] else torch.cat([y, z], -1)
    return torch.cat([turned, x[..., r:]], -1).to(torch.bfloat16)


def _tokens(s):
    """Each token's sequence, place in it and position."""
    tok = torch.arange(s["t"], device="cuda")
    cu, n = s["cu_q_lens"].long(), s["n"]
    seq = torch.searchsorted(cu[1:n + 1].contiguous(), tok, right=True)
    j = tok - cu[seq]
    return seq, j, s["kv_lens"].long()[seq] - (cu[seq + 1] - cu[seq]) + j


def _pack(x):
    """x [t, heads, d] bf16 -> the values two a byte [t, heads, d / 2], and their groups' s and m as bytes."""
    d = x.shape[-1]
    v = x.float().unflatten(-1, (-1, _group(d)))
    m = v.amin(-1, keepdim=True)
    s = ((v.amax(-1, keepdim=True) - m) / 15).bfloat16().float()
    n = torch.round((v - m) / torch.where(s > 0, s, torch.ones_like(s))).clamp(0, 15).flatten(-2).to(torch.uint8)
    return n[..., 0::2] | n[..., 1::2] << 4, torch.cat([s, m], -1).bfloat16().flatten(-2).view(torch.uint8)


def _unpack(row, d):
    """Rows [..., row_bytes] -> K and V [..., d] float32."""
    n = d // _group(d)
    v = torch.stack([row[..., :d] & 15, row[..., :d] >> 4], -1).flatten(-2).float()
    sm = row[..., d:d + 8 * n].contiguous().view(torch.bfloat16).float().unflatten(-1, (2 * n, 2))
    x = v.unflatten(-1, (2 * n, -1)) * sm[..., :1] + sm[..., 1:]
    return x[..., :n, :].flatten(-2), x[..., n:, :].flatten(-2)


def _store(s):
    c, t, d = s["case"], s["t"], s["case"]["d"]
    seq, _, pos = _tokens(s)
    slot = s["page_indices"][seq, pos // c["ps"]].long() * c["ps"] + pos % c["ps"]
    s["q_out"][:t] = _rotate(s, s["q"][:t], pos)
    (k, ks), (v, vs) = _pack(_rotate(s, s["k"][:t], pos)), _pack(s["v"][:t])
    flat = s["kv"].view(-1, c["hkv"], _row_bytes(d))
    flat[slot, :, :d + 8 * (d // _group(d))] = torch.cat([k, v, ks, vs], -1)
    back = _unpack(flat[slot], d)
    s["k_out"][:t], s["v_out"][:t] = back
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _probabilities(s, lo, hi, qm):
    """Softmax of sequences lo..hi (at most qm queries each): [m, hkv, g * qm, most], the keys' slots [m, most] and their values."""
    c, kv = s["case"], s["kv"]
    ps, hkv, d, hq = c["ps"], c["hkv"], c["d"], c["hq"]
    m, g = hi - lo, hq // hkv
    lens, cu = s["kv_lens"][lo:hi].long(), s["cu_q_lens"].long()
    key = torch.arange(s["most"], device="cuda")
    slot = (s["page_indices"][lo:hi].long()[:, :, None] * ps + torch.arange(ps, device="cuda")).flatten(1)
    x = kv.view(-1, *kv.shape[2:])[slot]
    k, v = _unpack(x, d) if kv.dtype == torch.uint8 else (x[:, :, 0::2].float(), None)
    tok = cu[lo:hi, None] + torch.arange(qm, device="cuda")
    q = s["q"][tok.clamp(max=s["q"].shape[0] - 1)].float().view(m, qm, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(m, hkv, g * qm, d)
    score = (q @ k.permute(0, 2, 3, 1)) * s["sm_scale"]
    if c["cap"]:
        score = c["cap"] * torch.tanh(score / c["cap"])
    at = lens[:, None] - (cu[lo + 1:hi + 1] - cu[lo:hi])[:, None] + torch.arange(qm, device="cuda")  # positions
    hidden = key > at[..., None]
    if c["window"]:
        hidden |= key <= at[..., None] - c["window"]
    score.masked_fill_(hidden.repeat(1, g, 1)[:, None], -math.inf)
    p = (score - score.amax(-1, keepdim=True)).exp_()
    return p.div_(p.sum(-1, keepdim=True)), slot, v


def _attend(s, lo, hi, qm):
    """Attention of sequences lo..hi: [m, qm, hq, d] float32."""
    c = s["case"]
    p, _, v = _probabilities(s, lo, hi, qm)
    o = p @ v.permute(0, 2, 1, 3)
    g = c["hq"] // c["hkv"]
    return o.unflatten(2, (g, qm)).permute(0, 3, 1, 2, 4).reshape(hi - lo, qm, c["hq"], c["d"])


def _add_weights(s, lo, hi, qm):
    """Writes the new weights of the keys of sequences lo..hi."""
    c, ps = s["case"], s["case"]["ps"]
    p, slot, _ = _probabilities(s, lo, hi, qm)
    new = p.sum(2)  # [m, hkv, most]
    real = (torch.arange(s["most"], device="cuda") < s["kv_lens"][lo:hi, None])
    at, w = slot[real], new.permute(0, 2, 1)[real]  # [keys], [keys, hkv]
    s["weights_out"][at // ps, :, at % ps] = c["keep"] * s["weights"][at // ps, :, at % ps] + w


def _evict(s):
    c, n, ps, hkv = s["case"], s["n"], s["case"]["ps"], s["case"]["hkv"]
    lens = s["kv_lens"][:n].long()
    keep = torch.minimum(lens, s["budgets"][:n].long().clamp(min=c["sinks"] + c["recent"]))[:, None, None]
    key = torch.arange(s["most"], device="cuda")
    pages = s["page_indices"][:n].long()
    w = s["weights"][pages].permute(0, 2, 1, 3).flatten(2)  # [n, hkv, most]
    real = (key < lens[:, None])[:, None]
    safe = ((key < c["sinks"]) | (key >= (lens - c["recent"])[:, None]))[:, None]
    order = w.masked_fill(safe, math.inf).masked_fill(~real, -math.inf).sort(dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(order, dtype=torch.bool).scatter_(-1, order, (key < keep).expand_as(order)) & real
    holes, movers = (~kept & (key < keep)).nonzero(), (kept & (key >= keep)).nonzero()
    place = key.expand(n, hkv, -1).clone()
    place[holes.unbind(1)] = movers[:, 2]
    slot = (pages[:, :, None] * ps + torch.arange(ps, device="cuda")).flatten(1)
    to, frm, h = slot[holes[:, 0], holes[:, 2]], slot[movers[:, 0], movers[:, 2]], holes[:, 1]
    flat = (s["kv"].view(torch.uint8) if s["kv"].dtype == E4M3 else s["kv"]).view(-1, hkv, 2 * c["d"])
    flat[to, h] = flat[frm, h]
    front = (key < keep).expand(n, hkv, -1)
    i, h, k = front.nonzero().unbind(1)
    at = slot[i, k]
    s["weights_out"][at // ps, h, at % ps] = w[i, h, place[front]]
    s["slots_out"][i, h, k] = place[front].int()
    s["lens_out"][:n] = keep[:, 0, 0].int()
    return {"lens": s["lens_out"], "slots": s["slots_out"], "weights": s["weights_out"], "kv": s["kv"]}


def _plain(s):
    c = s["case"]
    if c["op"] == "store":
        return _store(s)
    if c["op"] == "evict":
        return _evict(s)
    nd = c["nd"]
    if c["op"] == "attend":
        if nd:
            s["out"][:nd] = _attend(s, 0, nd, 1)[:, 0].to(torch.bfloat16)
        if c["nc"]:
            s["out"][nd:s["t"]] = _attend(s, nd, s["n"], c["cl"]).flatten(0, 1).to(torch.bfloat16)
        return {"out": s["out"]}
    if nd:
        _add_weights(s, 0, nd, 1)
    if c["nc"]:
        _add_weights(s, nd, s["n"], c["cl"])
    return {"weights": s["weights_out"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits
def _turned(c, x, positions):
    """float64 [t, heads, d] turned: each pair as a complex number times e^(i p f)."""
    r, f = c["rot"], []
    for i in range(r // 2):
        w = (500000.0 if c["scaling"] == "llama3" else 10000.0) ** (-2.0 * i / r)
        if c["scaling"] == "llama3":
            wave = 2.0 * math.pi / w
            if wave > 8192.0 / 1.0:
                w /= 8.0
            elif wave >= 8192.0 / 4.0:
                smooth = (8192.0 / wave - 1.0) / 3.0
                w = (1.0 - smooth) * w / 8.0 + smooth * w
        f.append(w)
    phase = positions.double()[:, None] * torch.tensor(f, dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.ones_like(phase), phase)[:, None, :]
    y = x.clone()
    if c["inter"]:
        y[..., :r] = torch.view_as_real(torch.view_as_complex(x[..., :r].unflatten(-1, (r // 2, 2)).contiguous()) * turn).flatten(-2)
    else:
        z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * turn
        y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
    return y


def _held(x):
    """float64 values of x [t, heads, d] (bf16 values) as the 4-bit rows stand for them."""
    size = 32 if x.shape[-1] == 64 else 64
    y = x.view(*x.shape[:-1], -1, size)
    least, greatest = y.min(-1, True).values, y.max(-1, True).values
    step = ((greatest - least) / 15.0).to(torch.bfloat16).double()
    level = torch.round((y - least) / step.clamp(min=1e-300)).clamp(0.0, 15.0)
    return (least + level * step).view(x.shape)


def _values(c, s, rows):
    """float64 K and V [keys, hkv, d] of cache rows."""
    d, hkv = c["d"], c["hkv"]
    if s["kv"].dtype != torch.uint8:
        x = s["kv"].view(-1, 2 * hkv, d)[rows].double()
        return x[:, 0::2], x[:, 1::2]
    x, size = s["kv"].view(-1, hkv, s["kv"].shape[-1])[rows], 32 if d == 64 else 64
    both = []
    for part in range(2):
        byte = x[..., part * d // 2:(part + 1) * d // 2].long()
        level = torch.empty(*byte.shape[:-1], d, dtype=torch.float64, device=byte.device)
        level[..., 0::2], level[..., 1::2] = (byte % 16).double(), (byte // 16).double()
        a = d + part * 4 * (d // size)
        pair = x[..., a:a + 4 * (d // size)].contiguous().view(torch.bfloat16).double()
        both.append(level * pair[..., 0::2].repeat_interleave(size, -1) + pair[..., 1::2].repeat_interleave(size, -1))
    return both


def exact(case, seed):
    c, s = case, prepare(case, seed)
    ql, kl = _lens(c)
    ps, hkv, d = c["ps"], c["hkv"], c["d"]
    pages = s["page_indices"].cpu().long()
    place = [(pages[i, :, None] * ps + torch.arange(ps)).flatten()[:k] for i, k in enumerate(kl)]  # each key's row
    if c["op"] == "evict":
        w, w_out = s["weights"].cpu().permute(0, 2, 1).reshape(-1, hkv).numpy(), s["weights_out"].cpu().double()
        lens_out, slots_out = s["lens_out"].cpu(), s["slots_out"].cpu()
        flat = (s["kv"].view(torch.uint8) if c["kv"] == "fp8" else s["kv"]).view(-1, hkv, 2 * d)
        for i, k in enumerate(kl):
            rows = place[i].numpy()
            keep = min(k, max(c["keep"], c["sinks"] + c["recent"]))
            lens_out[i] = keep
            for h in range(hkv):
                score = w[rows, h].astype(np.float64)
                score[:c["sinks"]] = np.inf
                score[max(0, k - c["recent"]):] = np.inf
                stay = np.zeros(k, bool)
                stay[np.lexsort((np.arange(k), -score))[:keep]] = True
                source = np.arange(keep)
                source[~stay[:keep]] = keep + np.flatnonzero(stay[keep:])
                changed = np.flatnonzero(~stay[:keep])
                if len(changed):
                    flat[torch.from_numpy(rows[changed]).cuda(), h] = flat[torch.from_numpy(rows[source[changed]]).cuda(), h]
                w_out[torch.from_numpy(rows[:keep] // ps), h, torch.from_numpy(rows[:keep] % ps)] = torch.from_numpy(w[rows[source], h].astype(np.float64))
                slots_out[i, h, :keep] = torch.from_numpy(source)
        return {"lens": lens_out, "slots": slots_out, "weights": w_out, "kv": s["kv"]}
    t = sum(ql)
    if c["op"] == "store":
        position = torch.cat([torch.arange(k - n, k) for n, k in zip(ql, kl)]).cuda()
        out = {x: torch.zeros(s[x + "_out"].shape, dtype=torch.float64, device="cuda") for x in "qkv"}
        out["q"][:t] = _turned(c, s["q"][:t].double(), position)
        out["k"][:t] = _held(_turned(c, s["k"][:t].double(), position).to(torch.bfloat16).double())
        out["v"][:t] = _held(s["v"][:t].double())
        return out
    g = c["hq"] // hkv
    starts = np.concatenate([[0], np.cumsum(ql)]).tolist()
    q = s["q"].double()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    new = s["weights_out"].double() if c["op"] == "weights" else None
    for i, (n, k) in enumerate(zip(ql, kl)):
        keys, values = _values(c, s, place[i].cuda())
        a = starts[i]
        at = torch.arange(k - n, k, device="cuda")[:, None]
        key = torch.arange(k, device="cuda")[None, :]
        hidden = (key > at) | (key <= at - c["window"]) if c["window"] else key > at
        for h in range(hkv):
            w = torch.einsum("qgd,kd->gqk", q[a:a + n, h * g:(h + 1) * g], keys[:, h]) * s["sm_scale"]
            if c["cap"]:
                w = torch.tanh(w / c["cap"]) * c["cap"]
            w = torch.softmax(w.masked_fill_(hidden, -math.inf), -1)
            if new is None:
                out[a:a + n, h * g:(h + 1) * g] = torch.einsum("gqk,kd->qgd", w, values[:, h])
            else:
                r = place[i].cuda()
                new[r // ps, h, r % ps] = c["keep"] * s["weights"].double()[r // ps, h, r % ps] + w.sum((0, 1))
    return {"out": out} if new is None else {"weights": new}
