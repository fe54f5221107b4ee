"""Key weights and eviction on the GPU against their float64 forms, and the operators of a long context together: 4-bit rows
written, attended to, weighed and thinned out, step after step."""
import math

import numpy as np
import pytest
import torch

from long_context import BF16, Batch, pack_rows, row_bytes, unpack_rows
from ragged_paged_attention_gb300 import api

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn
LENS = ([1, 3, 0, 2, 40, 1, 300, 17, 5], [1, 700, 64, 2, 40, 1500, 1300, 17, 2000])


def weigh(b, old, keep, in_place=False, **kw):
    kv, lens, pages, cu, num = b.gpu()
    q, w = b.q.cuda(), None if old is None else old.cuda()
    prm = api._batch_params(q.get_device(), *q.shape, kv, lens, pages, cu, num, g4=b.g4)
    ws = torch.zeros(api.rpa_key_weights_workspace_size(prm), dtype=torch.uint8, device="cuda")
    out = w if in_place else torch.full((b.total, b.hkv, b.ps), -3.0, device="cuda")
    got = api.rpa_key_weights(q, kv, lens, pages, cu, num, w, keep=keep, weights_out=None if in_place else out, workspace=ws, **kw)
    assert got is out
    return out.cpu(), api.check_device_status(ws)


def check_weights(b, *, keep=0.75, in_place=False, seed=0, **kw):
    kw.setdefault("sm_scale", b.d ** -0.5)
    g = torch.Generator().manual_seed(seed)
    old = torch.rand(b.total, b.hkv, b.ps, generator=g)
    got, bits = weigh(b, None if keep == 0.0 else old, keep, in_place, **kw)
    assert bits == 0, hex(bits)
    want = (old.clone() if in_place else torch.full_like(old, -3.0)).double()
    size = torch.zeros_like(want)
    for i, n in enumerate(b.q_lens):
        if n == 0:
            continue
        new = b.probabilities(i, kw["sm_scale"], kw.get("sliding_window"), kw.get("soft_cap"))
        new = new.unflatten(0, (b.hkv, -1)).sum((1, 2)).T  # [keys, hkv]
        at = b.place[i]
        want[at // b.ps, :, at % b.ps] = (keep * old[at // b.ps, :, at % b.ps].double() if keep else 0.0) + new
        size[at // b.ps, :, at % b.ps] = new
    # A score is a sum of d exact products in float32, each addition within 2^-24 of a partial sum of at most sum |q k|,
    # about 0.64 d for unit values and scale |.| in all; times log2(e), exponentiated within 2^-22 and divided by a sum
    # of such terms: twice (d + 8) 2^-24 (0.64 d |sm_scale|) + 2^-20 of a probability, if every rounding went one way
    rel = 2 * (b.d + 8) * 2.0 ** -24 * 0.64 * b.d * abs(kw["sm_scale"]) + 2.0 ** -20
    if kw.get("soft_cap"):
        rel += 2 * 2.0 ** -21 * abs(kw["soft_cap"])  # tanhf: 2 units in the last place, times the cap
    err = (got.double() - want).abs()
    assert (err <= rel * size + 2.0 ** -23 * want.abs()).all(), ((err - 2.0 ** -23 * want.abs()) / size.clamp(min=1e-30)).max()
    assert err.norm() <= 1e-5 * (size.norm() + 1e-30) + 2.0 ** -24 * want.norm()
    return got


@pytest.mark.parametrize("g4", [False, True])
@pytest.mark.parametrize("hq,hkv,d,ps", [(4, 4, 64, 16), (8, 2, 128, 16), (4, 2, 256, 32), (6, 1, 128, 8), (3, 3, 64, 12),
                                         (16, 1, 128, 128), (24, 2, 64, 1)])
def test_weights_of_ragged_batches(hq, hkv, d, ps, g4):
    check_weights(Batch(*LENS, hq, hkv, d, ps, g4=g4, seed=hq + d))


@pytest.mark.parametrize("g4", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kw", [dict(keep=0.0), dict(keep=1.0, in_place=True), dict(sliding_window=1), dict(sliding_window=130),
                                dict(soft_cap=5.0), dict(soft_cap=30.0, sliding_window=500), dict(sm_scale=-0.125),
                                dict(sm_scale=1.0), dict(sm_scale=0.0)], ids=str)
def test_options_of_the_weights(kw, d, g4):
    check_weights(Batch(*LENS, 8, 2, d, 16, g4=g4, seed=d), **kw)


@pytest.mark.parametrize("g4", [False, True])
@pytest.mark.parametrize("q_lens,kv_lens", [([1] * 40, list(range(1, 3000, 75))), ([1], [30000]), ([1, 1], [1, 2]), ([1], [16]),
                                            ([129], [129]), ([32] * 3, [4000, 32, 513]), ([0, 0], [5, 0]), ([700], [2000])])
def test_weights_of_batch_shapes(q_lens, kv_lens, g4):
    check_weights(Batch(q_lens, kv_lens, 8, 2, 128, 16, g4=g4, seed=len(q_lens)))


@pytest.mark.parametrize("hq,hkv", [(12, 2), (40, 8), (48, 1), (71, 1), (130, 1), (160, 1)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_weights_of_group_sizes(hq, hkv, d):
    check_weights(Batch([1, 3, 0, 2, 40, 1, 30], [1, 700, 64, 2, 40, 600, 330], hq, hkv, d, 16, seed=hq), sliding_window=200 if hq == 40 else None)


@pytest.mark.parametrize("g4", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("scale,cap", [(-0.2, 20.0), (0.0, 5.0), (0.3, 1.5), (-0.1, None), (0.0, None)])
def test_weights_with_any_scale_and_cap(scale, cap, d, g4):
    check_weights(Batch([1, 40, 2, 150], [900, 300, 70, 1200], 8, 2, d, 16, g4=g4, seed=d), sm_scale=scale, soft_cap=cap)


@pytest.mark.parametrize("g4", [False, True])
def test_weights_of_many_sequences(g4):
    g = torch.Generator().manual_seed(5)
    q_lens = torch.randint(0, 3, (2500,), generator=g)
    kv_lens = q_lens + torch.randint(0, 40, (2500,), generator=g)
    check_weights(Batch(q_lens.tolist(), kv_lens.tolist(), 4, 2, 64, 16, g4=g4, seed=6))


def test_weights_add_up_over_calls():
    b = Batch(*LENS, 8, 2, 128, 16, seed=3)
    zero = torch.zeros(b.total, b.hkv, b.ps)
    once, _ = weigh(b, zero, 1.0, sm_scale=0.1)
    twice, _ = weigh(b, torch.where(once < 0, zero, once), 1.0, sm_scale=0.1)
    real = once >= 0
    assert ((twice - 2 * once).abs()[real] <= 2.0 ** -22 * once[real]).all()
    # every query gives 1 in all
    total = sum(n * b.hq for n in b.q_lens)
    assert abs(float(once[real].double().sum()) - total) <= 1e-5 * total


@pytest.mark.parametrize("g4", [False, True])
def test_weights_refuse_bad_metadata_on_the_device(g4):
    for change, bit in (("page", 0x08), ("q", 0x02), ("kv", 0x04), ("tokens", 0x10), ("num", 0x01), ("again", 0x10)):
        b = Batch([1, 20, 1], [300, 500, 40], 8, 2, 128, 16, g4=g4, seed=3)
        if change == "page":
            b.table[1, 3] = b.total
        elif change == "q":
            b.kv_lens[1] = 19
        elif change == "kv":
            b.kv_lens[1] = b.table.shape[1] * 16 + 1
        elif change == "tokens":
            b.cu[2:4] = torch.tensor([10 ** 6, 10 ** 6 + 1])
        elif change == "again":
            b.cu[:4] = torch.tensor([0, 22, 0, 22])
        else:
            b.num[0] = 9
        got, bits = weigh(b, torch.zeros(b.total, 2, 16), 1.0, sm_scale=0.1)
        assert bits & bit, (change, bits)
        if change in ("q", "kv"):
            at = b.place[1]
            assert (got[at // 16, :, at % 16] == -3.0).all()
        if change == "num":
            assert (got == -3.0).all()


# ------------------------------------------------------------------ eviction
def evict_plainly(kv_rows, weights, place, ps, budget, sinks, recent):
    """(new length, source slots [hkv, new length], kv_rows after) of one sequence; kv_rows [slots, hkv, bytes]."""
    n, hkv = len(place), kv_rows.shape[1]
    keep = min(n, max(budget, sinks + recent))
    source, rows = [], kv_rows.clone()
    for h in range(hkv):
        w = weights[place // ps, h, place % ps].double().numpy().copy()
        w[np.isnan(w)] = -math.inf
        nan = torch.isnan(weights[place // ps, h, place % ps]).numpy()
        first = np.zeros(n, bool)
        first[:sinks] = True
        first[max(0, n - recent):] = True
        order = sorted(range(n), key=lambda i: (not first[i], nan[i] and not first[i], 0.0 if first[i] else -w[i], i))
        stay = np.zeros(n, bool)
        stay[order[:keep]] = True
        src = np.arange(keep)
        src[~stay[:keep]] = keep + np.flatnonzero(stay[keep:])
        source.append(src)
        rows[place[:keep], h] = kv_rows[place[torch.from_numpy(src)], h]
    return keep, np.stack(source), rows


def cache_rows(b):
    """The cache as [slots, hkv, bytes]."""
    return b.kv.view(torch.uint8).reshape(b.total * b.ps, b.hkv, -1)


def check_evict(b, weights, budgets, max_keys, *, sinks=0, recent=0, in_place=False):
    n = len(b.lens)
    kv, lens, pages, _, num = b.gpu()
    w = weights.cuda()
    bud = torch.tensor(list(budgets) + [0] * (len(b.kv_lens) - n), dtype=torch.int32, device="cuda")
    prm = api.make_evict_params(kv, pages, max_keys, sinks=sinks, recent=recent)
    ws = torch.zeros(api.rpa_evict_workspace_size(prm), dtype=torch.uint8, device="cuda")
    w_out = w if in_place else torch.full_like(w, -3.0)
    lens_out = lens if in_place else torch.full_like(lens, -5)
    slots = torch.full((len(b.kv_lens), b.hkv, max_keys), -9, dtype=torch.int32, device="cuda")
    got = api.rpa_evict_kv_cache(kv, lens, pages, num, w, bud, max_keys, sinks=sinks, recent=recent, kv_lens_out=lens_out,
                                 slots_out=slots, weights_out=w_out, workspace=ws)
    assert got[0] is lens_out and got[1] is slots and api.check_device_status(ws) == 0
    rows, want_w = cache_rows(b), (weights.clone() if in_place else torch.full_like(weights, -3.0))
    for i in range(n):
        keep, source, rows = evict_plainly(rows, weights, b.place[i], b.ps, budgets[i], sinks, recent)
        assert int(lens_out[i]) == keep
        assert np.array_equal(slots[i, :, :keep].cpu().numpy(), source)
        assert (slots[i, :, keep:] == -9).all()
        at = b.place[i]
        for h in range(b.hkv):
            want_w[at[:keep] // b.ps, h, at[:keep] % b.ps] = weights[at[source[h]] // b.ps, h, at[source[h]] % b.ps]
    assert torch.equal(kv.cpu().view(torch.uint8).reshape(rows.shape), rows)
    assert torch.equal(w_out.cpu().nan_to_num(7.7), want_w.nan_to_num(7.7))
    assert torch.equal(lens_out[n:].cpu(), b.kv_lens[n:] if in_place else torch.full((len(b.kv_lens) - n,), -5, dtype=torch.int32))


def random_weights(b, seed=0, power=6):
    g = torch.Generator().manual_seed(seed)
    return torch.rand(b.total, b.hkv, b.ps, generator=g) ** power


EVICT = [1, 5, 0, 700, 64, 1500, 1300, 17, 2000], [0, 5, 3, 200, 64, 1499, 1, 100, 1000]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("g4,dtype", [(True, None), (False, BF16), (False, FP8), (False, torch.int8)], ids=str)
@pytest.mark.parametrize("hkv,d,ps", [(4, 64, 16), (2, 128, 16), (1, 256, 32), (3, 64, 12), (8, 128, 1)])
def test_evict(hkv, d, ps, g4, dtype, in_place):
    lens, budgets = EVICT
    b = Batch([0] * len(lens), lens, hkv, hkv, d, ps, g4=g4, dtype=dtype or BF16, seed=d)
    check_evict(b, random_weights(b, d), budgets, 1600, sinks=2, recent=7, in_place=in_place)


@pytest.mark.parametrize("sinks,recent", [(0, 0), (4, 0), (0, 64), (300, 300), (1, 1599)])
def test_keys_that_always_stay(sinks, recent):
    lens, budgets = EVICT
    b = Batch([0] * len(lens), lens, 2, 2, 128, 16, seed=1)
    check_evict(b, random_weights(b, 1), budgets, 1600, sinks=sinks, recent=recent)


@pytest.mark.parametrize("values", ["equal", "few", "signs", "odd", "ascending", "descending"])
def test_orders_of_weights(values):
    lens, budgets = EVICT
    b = Batch([0] * len(lens), lens, 2, 2, 64, 16, seed=2)
    w = random_weights(b, 3, 1)
    if values == "equal":
        w = torch.full_like(w, 0.25)
    elif values == "few":
        w = (w * 4).floor()
    elif values == "signs":
        w = (w - 0.5) * 1e3
        w[w.abs() < 300] = 0.0
        w[::2][w[::2] == 0] = -0.0
    elif values == "odd":
        w[w < 0.2] = math.nan
        w[(w > 0.2) & (w < 0.3)] = -math.inf
        w[w > 0.9] = math.inf
        w[(w > 0.5) & (w < 0.6)] *= 2.0 ** -140
    else:
        for at in b.place:
            w[at // 16, :, at % 16] = torch.arange(len(at), dtype=torch.float32)[:, None] * (1 if values == "ascending" else -1)
    check_evict(b, w, budgets, 1600, sinks=1, recent=3)


@pytest.mark.parametrize("n", [20000, 60000])
def test_evict_long_sequences(n):
    # (60000 keys are more than a block holds in shared memory)
    b = Batch([0, 0], [n, 1000], 2, 2, 64, 16, seed=4)
    check_evict(b, random_weights(b, 5), [n // 3, 1000], n, sinks=4, recent=200)


def test_evict_many_sequences():
    g = torch.Generator().manual_seed(7)
    lens = torch.randint(0, 60, (700,), generator=g).tolist()
    b = Batch([0] * 700, lens, 2, 2, 64, 8, seed=8)
    check_evict(b, random_weights(b, 9), torch.randint(0, 61, (700,), generator=g).tolist(), 60)


def test_evict_leaves_bad_sequences_alone():
    for change, bit in (("page", 0x08), ("kv", 0x04), ("budget", 0x100), ("negative", 0x100), ("num", 0x01)):
        b = Batch([0] * 3, [300, 500, 40], 2, 2, 128, 16, seed=3)
        kv, lens, pages, _, num = b.gpu()
        bud = torch.tensor([100, 100, 10, 0], dtype=torch.int32, device="cuda")
        if change == "page":
            pages[1, 3] = b.total
        elif change == "kv":
            lens[1] = pages.shape[1] * 16 + 1
        elif change == "budget":
            bud[1] = 201
        elif change == "negative":
            bud[1] = -1
        else:
            num[0] = 9
        ws = torch.zeros(api.rpa_evict_workspace_size(api.make_evict_params(kv, pages, 200)), dtype=torch.uint8, device="cuda")
        before, old = kv.clone(), lens.clone()
        out, slots = api.rpa_evict_kv_cache(kv, lens, pages, num, random_weights(b).cuda(), bud, 200, workspace=ws)
        assert api.check_device_status(ws) == bit, change
        rows, was = (x.view(torch.uint8).reshape(b.total * 16, -1)[b.place[1]] for x in (kv, before))
        assert torch.equal(rows, was) and int(out[1]) == int(old[1])
        assert int(out[0]) == (300 if change == "num" else 100)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_long_context_kept_short(d):
    # prompts written into a 4-bit cache and attended to, their last queries weighing the keys; then decode steps that write,
    # attend, add weights and cut back: every step against float64 on the cache's own bytes
    hq, hkv, ps, n = 8, 2, 16, 3
    g = torch.Generator().manual_seed(d)
    lens, budget, pps = [300, 45, 160], 96, 24
    table = torch.arange(n * pps, dtype=torch.int32).flip(0).reshape(n, pps).cuda()
    pages = n * pps
    kv = torch.zeros(pages, ps, hkv, row_bytes(d), dtype=torch.uint8, device="cuda")
    w = torch.zeros(pages, hkv, ps, device="cuda")
    num = torch.tensor([n], dtype=torch.int32, device="cuda")
    rope, scale = api.make_rope_table(d), d ** -0.5
    randn = lambda *s: torch.randn(*s, generator=g).to(BF16).cuda()  # noqa: E731
    batch = lambda ql: torch.tensor([0] + np.cumsum(ql).tolist(), dtype=torch.int32, device="cuda")  # noqa: E731

    def values(i, m):
        slot = (table[i, :, None].long() * ps + torch.arange(ps, device="cuda")).flatten()[:m]
        return unpack_rows(kv.flatten(0, 1)[slot].cpu(), d), slot

    def softmax(q, i, m):  # q [q, hq, d], the last of the sequence's m keys
        k = values(i, m)[0][0].repeat_interleave(hq // hkv, 1)
        s = torch.einsum("qhd,khd->hqk", q.double().cpu(), k) * scale
        hidden = torch.arange(m)[None] > torch.arange(m - len(q), m)[:, None]
        return torch.softmax(s.masked_fill(hidden, -math.inf), -1)

    ql, now = list(lens), list(lens)
    position = list(lens)  # the tokens so far, whatever the cache has kept
    for step in range(6):
        t, cu = sum(ql), batch(ql)
        kv_lens = torch.tensor(now, dtype=torch.int32, device="cuda")
        q, k, v = randn(t, hq, d), randn(t, hkv, d), randn(t, hkv, d)
        pos = torch.cat([torch.arange(p - m, p) for p, m in zip(position, ql)]).int().cuda()
        q, _ = api.rpa_g4_update_kv_cache(q, k, v, kv, kv_lens, table, cu, num, rope, positions=pos)
        out = api.rpa_g4_forward(q, kv, kv_lens, table, cu, num, sm_scale=scale)
        back_k, back_v = api.rpa_g4_read_kv_cache(kv, kv_lens, table, cu, num, t)
        tail = [min(m, 8) for m in ql]  # the queries that weigh
        qs = torch.cat([q[cu[i + 1] - m:cu[i + 1]] for i, m in enumerate(tail)])
        before = w.clone()
        api.rpa_key_weights(qs, kv, kv_lens, table, batch(tail), num, w, sm_scale=scale)
        torch.cuda.synchronize()
        for i in range(n):
            a, e = int(cu[i]), int(cu[i + 1])
            (keys, vals), slot = values(i, now[i])
            p = softmax(q[a:e], i, now[i])
            want = torch.einsum("hqk,khd->qhd", p, vals.repeat_interleave(hq // hkv, 1))
            assert (out[a:e].double().cpu() - want).norm() <= 5e-3 * want.norm()
            assert torch.equal(back_k[a:e].cpu(), keys[now[i] - ql[i]:].float().to(BF16))
            assert torch.equal(back_v[a:e].cpu(), vals[now[i] - ql[i]:].float().to(BF16))
            new = p[:, -tail[i]:].unflatten(0, (hkv, -1)).sum((1, 2)).T
            got = (w - before)[slot // ps, :, slot % ps].cpu().double()
            assert (got - new).norm() <= 1e-5 * new.norm() + 1e-6
        budgets = torch.full((n,), budget, dtype=torch.int32, device="cuda")
        new_lens, slots = api.rpa_evict_kv_cache(kv, kv_lens, table, num, w, budgets, budget, sinks=2, recent=16, kv_lens_out=kv_lens,
                                                 weights_out=w)
        assert new_lens is kv_lens
        now = kv_lens.tolist()
        assert now == [min(budget, m) for m in [x for x in (lens if step == 0 else lens_before)]]
        for i in range(n):
            assert torch.equal(slots[i, :, :2].cpu(), torch.tensor([[0, 1]] * hkv, dtype=torch.int32))
        ql = [1, 3, 2]
        position = [p + m for p, m in zip(position, ql)]
        now = [m + x for m, x in zip(now, ql)]
        lens_before = list(now)
        # the slots of new tokens start without weight
        for i in range(n):
            slot = (table[i, :, None].long() * ps + torch.arange(ps, device="cuda")).flatten()[now[i] - ql[i]:now[i]]
            w[slot // ps, :, slot % ps] = 0.0


@pytest.mark.parametrize("g4", [False, True])
def test_captured_weights_and_eviction_replay(g4):
    b = Batch([1, 3, 40, 1], [100, 700, 300, 1], 8, 2, 128, 16, g4=g4, seed=1)
    kv, lens, pages, cu, num = b.gpu()
    q, w = b.q.cuda(), random_weights(b).cuda()
    budgets = torch.full((len(b.kv_lens),), 80, dtype=torch.int32, device="cuda")

    def call(cache):
        new = api.rpa_key_weights(q, cache, lens, pages, cu, num, w, sm_scale=0.1, weights_out=torch.zeros_like(w))
        new_lens, slots = api.rpa_evict_kv_cache(cache, lens, pages, num, new, budgets, 80, sinks=1, recent=5,
                                                 slots_out=torch.zeros(len(b.kv_lens), 2, 80, dtype=torch.int32, device="cuda"))
        return new, new_lens, slots

    call(kv.clone())
    torch.cuda.synchronize()
    mine = kv.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(mine)
    for m in ([100, 700, 300, 1], [90, 81, 79, 1]):
        lens[:4] = torch.tensor(m, dtype=torch.int32).cuda()
        mine.copy_(kv)
        graph.replay()
        other = kv.clone()
        want = call(other)
        for x, y in zip(out, want):
            assert torch.equal(x, y)
        assert torch.equal(mine.view(torch.uint8), other.view(torch.uint8))
