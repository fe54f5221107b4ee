"""Eviction step after step on the GPU: what stays by when it came, against a plain form on the host. All comparisons are exact."""
import numpy as np
import pytest
import torch

from long_context import BF16, Batch, row_bytes
from ragged_paged_attention_gb300 import api
from test_gpu_long_context import cache_rows, check_evict, random_weights

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn
LENS, BUDGETS = [1, 5, 0, 700, 64, 1500, 1300, 17, 2000], [0, 5, 3, 200, 64, 1499, 1, 100, 1000]


def numbers_of(entries):
    """[n] entries of a sequence's head -> its keys' numbers: the new ones' (below 0) go on behind the greatest, slot by slot."""
    x = entries.astype(np.int64)
    new = np.flatnonzero(x < 0)
    if len(new):
        x[new] = x.max(initial=-1, where=x >= 0) + 1 + new - new[0]
    return x


def stays(weights, numbers, keep, sinks, recent):
    """Which of a head's keys stay: the first `sinks` slots and the last `recent` numbers, then by weight, then by slot."""
    n = len(weights)
    first = (np.arange(n) < sinks) | (numbers > (numbers.max() if n else 0) - recent)
    nan = np.isnan(weights) & ~first
    order = np.lexsort((np.arange(n), np.where(first | nan, 0.0, -weights), nan, ~first))
    stay = np.zeros(n, bool)
    stay[order[:keep]] = True
    return stay


def check(b, weights, budgets, max_keys, positions, *, sinks=0, recent=0, in_place=False):
    n = len(b.lens)
    kv, lens, pages, _, num = b.gpu()
    w, came = weights.cuda(), positions.cuda()
    bud = torch.tensor(list(budgets) + [0] * (len(b.kv_lens) - n), dtype=torch.int32, device="cuda")
    ws = torch.zeros(api.rpa_evict_workspace_size(api.make_evict_params(kv, pages, max_keys, sinks=sinks, recent=recent)),
                     dtype=torch.uint8, device="cuda")
    w_out = w if in_place else torch.full_like(w, -3.0)
    lens_out, slots = api.rpa_evict_kv_cache(kv, lens, pages, num, w, bud, max_keys, sinks=sinks, recent=recent,
                                             kv_lens_out=lens if in_place else None, weights_out=w_out, positions=came, workspace=ws)
    assert api.check_device_status(ws) == 0
    rows, want_came = cache_rows(b).clone(), positions.clone()
    want_w = weights.clone() if in_place else torch.full_like(weights, -3.0)
    before = rows.clone()
    for i in range(n):
        at, m = b.place[i], b.lens[i]
        keep = min(m, max(budgets[i], sinks + recent))
        assert int(lens_out[i]) == keep
        for h in range(b.hkv):
            numbers = numbers_of(positions[at // b.ps, h, at % b.ps].numpy())
            stay = stays(weights[at // b.ps, h, at % b.ps].double().numpy(), numbers, keep, sinks, recent)
            src = np.arange(keep)
            src[~stay[:keep]] = keep + np.flatnonzero(stay[keep:])
            assert np.array_equal(slots[i, h, :keep].cpu().numpy(), src), (i, h)
            rows[at[:keep], h] = before[at[src], h]
            want_w[at[:keep] // b.ps, h, at[:keep] % b.ps] = weights[at[src] // b.ps, h, at[src] % b.ps]
            want_came[at[:keep] // b.ps, h, at[:keep] % b.ps] = torch.from_numpy(numbers[src]).int()
            want_came[at[keep:] // b.ps, h, at[keep:] % b.ps] = -1
            want_w[at[keep:] // b.ps, h, at[keep:] % b.ps] = 0.0
    assert torch.equal(kv.cpu().view(torch.uint8).reshape(rows.shape), rows)
    assert torch.equal(w_out.cpu(), want_w) and torch.equal(came.cpu(), want_came)


def entries(b, kind, seed=0):
    """positions [pages, hkv, page_size]; slots that are no key's hold numbers that would come first."""
    g = torch.Generator().manual_seed(seed)
    x = torch.full((b.total, b.hkv, b.ps), 2 ** 30, dtype=torch.int32)
    for at in b.place:
        for h in range(b.hkv):
            m = len(at)
            v = torch.full((m,), -1, dtype=torch.int32)
            if kind == "grown" and m:  # cut before, with a few new keys behind
                old = m - min(m, 5)
                v[:old] = torch.randperm(3 * m, generator=g)[:old].int()
            elif kind == "all":
                v = (torch.randperm(5 * m, generator=g)[:m] * 7).int()
            elif kind == "gaps":       # new keys between others
                v = torch.randperm(2 * m, generator=g)[:m].int()
                v[torch.rand(m, generator=g) < 0.3] = -7
            x[at // b.ps, h, at % b.ps] = v
    return x


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["new", "grown", "all", "gaps"])
@pytest.mark.parametrize("hkv,d,ps,g4,dtype", [(4, 64, 16, True, BF16), (2, 128, 16, False, BF16), (1, 256, 32, False, FP8),
                                               (3, 64, 12, False, torch.int8), (8, 128, 1, True, BF16)], ids=str)
def test_recent_keys_by_when_they_came(hkv, d, ps, g4, dtype, kind, in_place):
    b = Batch([0] * len(LENS), LENS, hkv, hkv, d, ps, g4=g4, dtype=dtype, seed=d)
    check(b, random_weights(b, d), BUDGETS, 1600, entries(b, kind, ps), sinks=2, recent=7, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("hkv,d,ps", [(4, 64, 16), (3, 96, 12), (2, 128, 16), (1, 192, 8), (2, 256, 1)])
def test_int4_caches(hkv, d, ps, in_place):
    # (a row is d / 2 bytes of K and as many of V)
    b = Batch([0] * len(LENS), LENS, hkv, hkv, d // 2, ps, g4=False, dtype=torch.int8, seed=d)
    b.kv = b.kv.view(torch.uint8)
    check_evict(b, random_weights(b, d), BUDGETS, 1600, sinks=2, recent=7, in_place=in_place)
    check(b, random_weights(b, d), BUDGETS, 1600, entries(b, "grown", d), sinks=2, recent=7, in_place=in_place)


@pytest.mark.parametrize("sinks,recent", [(0, 0), (4, 0), (0, 64), (300, 300), (1, 1599)])
@pytest.mark.parametrize("kind", ["new", "grown", "gaps"])
def test_numbers_of_keys_that_always_stay(kind, sinks, recent):
    b = Batch([0] * len(LENS), LENS, 2, 2, 128, 16, seed=1)
    check(b, random_weights(b, 1), BUDGETS, 1600, entries(b, kind), sinks=sinks, recent=recent)


@pytest.mark.parametrize("n", [20000, 60000])
def test_numbers_of_long_sequences(n):
    # (60000 keys are more than a block holds in shared memory)
    b = Batch([0, 0], [n, 1000], 2, 2, 64, 16, seed=4)
    check(b, random_weights(b, 5), [n // 3, 1000], n, entries(b, "gaps"), sinks=4, recent=200)


def test_a_sequence_left_alone_keeps_its_entries():
    b = Batch([0] * 3, [300, 500, 40], 2, 2, 128, 16, seed=3)
    kv, lens, pages, _, num = b.gpu()
    pages[1, 3] = b.total
    came = entries(b, "gaps").cuda()
    before, w = came.clone(), random_weights(b).cuda()
    bud = torch.full((4,), 20, dtype=torch.int32, device="cuda")
    ws = torch.zeros(api.rpa_evict_workspace_size(api.make_evict_params(kv, pages, 40)), dtype=torch.uint8, device="cuda")
    api.rpa_evict_kv_cache(kv, lens, pages, num, w, bud, 40, recent=8, positions=came, workspace=ws)
    assert api.check_device_status(ws) == 0x08
    at = b.place[1]
    assert torch.equal(came.cpu()[at // 16, :, at % 16], before.cpu()[at // 16, :, at % 16])
    assert not torch.equal(came, before)


class Loop:
    """Sequences of a bf16 cache whose rows hold the tokens' numbers, growing by a few tokens a step and cut every step."""

    def __init__(self, lens, hkv=2, d=64, ps=16, pps=40):
        self.lens, self.count, self.hkv, self.ps, n = list(lens), list(lens), hkv, ps, len(lens)
        self.table = torch.arange(n * pps, dtype=torch.int32).flip(0).reshape(n, pps).cuda()
        self.kv = torch.zeros(n * pps, ps, 2 * hkv, d, dtype=BF16, device="cuda")
        self.w = torch.rand(n * pps, hkv, ps, generator=torch.Generator().manual_seed(1)).cuda()
        self.came = torch.full((n * pps, hkv, ps), -1, dtype=torch.int32, device="cuda")
        self.num = torch.tensor([n], dtype=torch.int32, device="cuda")
        for i, m in enumerate(lens):
            self.write(i, 0, list(range(m)))

    def slots(self, i, a, e):
        at = torch.arange(a, e, device="cuda")
        return self.table[i][at // self.ps].long(), at % self.ps

    def write(self, i, slot, tokens):
        page, at = self.slots(i, slot, slot + len(tokens))
        rows = self.kv.view(torch.int32).view(*self.kv.shape[:2], self.hkv, -1)  # [pages, ps, hkv, words of K and V]
        rows[page, at] = torch.tensor(tokens, dtype=torch.int32, device="cuda")[:, None, None]

    def tokens(self, i):
        """[hkv, keys] the tokens held."""
        page, at = self.slots(i, 0, self.lens[i])
        x = self.kv.view(torch.int32).view(*self.kv.shape[:2], self.hkv, -1)[page, at]
        assert (x == x[..., :1]).all()
        return x[..., 0].T.cpu()

    def cut(self, budget, **kw):
        lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        bud = torch.full((len(self.lens),), budget, dtype=torch.int32, device="cuda")
        api.rpa_evict_kv_cache(self.kv, lens, self.table, self.num, self.w, bud, budget, kv_lens_out=lens, weights_out=self.w,
                               positions=self.came, **kw)
        self.lens = lens.tolist()

    def grow(self, i, n):
        self.write(i, self.lens[i], list(range(self.count[i], self.count[i] + n)))
        self.lens[i] += n
        self.count[i] += n


def test_the_newest_keys_are_there_at_every_step():
    # new keys weigh least, so that none but `recent` would stay for its weight
    loop, budget, sinks, recent = Loop([500, 130, 97, 40]), 96, 3, 32
    for step in range(120):
        loop.w *= 1.01
        before = list(loop.lens)
        loop.cut(budget, sinks=sinks, recent=recent)
        for i, c in enumerate(loop.count):
            held, m = loop.tokens(i), loop.lens[i]
            assert m == min(budget, c)
            page, at = loop.slots(i, 0, m)
            assert torch.equal(loop.came[page, :, at].T.cpu(), held)
            for h in range(loop.hkv):
                assert len(set(held[h].tolist())) == m
                assert set(range(max(0, c - recent), c)) | set(range(min(c, sinks))) <= set(held[h].tolist()), (step, i, h)
            n = 1 + (step + i) % 3
            page, at = loop.slots(i, m, before[i])
            assert (loop.came[page, :, at] == -1).all() and (loop.w[page, :, at] == 0.0).all()
            loop.grow(i, n)


def test_new_tokens_start_without_weight():
    # a decode loop of key weights and eviction, nothing done by hand between: what each key holds is what it got itself
    hq, hkv, d, ps, pps, budget = 4, 2, 64, 16, 10, 48
    g = torch.Generator().manual_seed(2)
    count, lens = [60, 30], [60, 30]
    table = torch.arange(2 * pps, dtype=torch.int32).reshape(2, pps).cuda()
    kv = torch.randn(2 * pps, ps, 2 * hkv, d, generator=g).to(BF16).cuda()  # (every slot has had a key before)
    w = torch.zeros(2 * pps, hkv, ps, device="cuda")
    came = torch.full(w.shape, -1, dtype=torch.int32, device="cuda")
    num, cu = torch.tensor([2], dtype=torch.int32, device="cuda"), torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    got = [[{} for _ in range(hkv)] for _ in range(2)]  # each token's weight so far, float64
    held = [[list(range(m)) for _ in range(hkv)] for m in lens]
    for step in range(40):
        q = torch.randn(2, hq, d, generator=g).to(BF16).cuda()
        kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        api.rpa_key_weights(q, kv, kv_lens, table, cu, num, w, sm_scale=d ** -0.5)
        for i, m in enumerate(lens):
            at = (table[i, :, None].long() * ps + torch.arange(ps, device="cuda")).flatten()[:m]
            keys = kv.flatten(0, 1)[at][:, 0::2].double()
            p = torch.softmax(torch.einsum("hgd,khd->hgk", q[i].double().unflatten(0, (hkv, -1)), keys) * d ** -0.5, -1).sum(1).cpu()
            now = w[at // ps, :, at % ps].T.double().cpu()
            for h in range(hkv):
                for j, token in enumerate(held[i][h]):
                    got[i][h][token] = got[i][h].get(token, 0.0) + float(p[h, j])
                want = torch.tensor([got[i][h][t] for t in held[i][h]], dtype=torch.float64)
                # a score is a sum of d exact products in float32, each addition within 2^-24 of a partial sum of at most sum
                # |q k|, about 0.64 d, times the scale; exponentiated within 2^-22 and divided by a sum of such terms: twice
                # that of a share. Each step's sum is rounded to 2^-24 of itself
                rel = 2 * (d + 8) * 2.0 ** -24 * 0.64 * d ** 0.5 + 2.0 ** -20 + (step + 1) * 2.0 ** -24
                assert ((now[h] - want).abs() <= rel * want).all(), step
        bud = torch.full((2,), budget, dtype=torch.int32, device="cuda")
        _, slots = api.rpa_evict_kv_cache(kv, kv_lens, table, num, w, bud, budget, sinks=2, recent=8, kv_lens_out=kv_lens, weights_out=w,
                                          positions=came)
        lens = kv_lens.tolist()
        for i in range(2):
            held[i] = [[held[i][h][j] for j in slots[i, h, :lens[i]].tolist()] + [count[i]] for h in range(hkv)]
            kv.flatten(0, 1)[int(table[i, lens[i] // ps]) * ps + lens[i] % ps] = torch.randn(2 * hkv, d, generator=g).to(BF16).cuda()
            lens[i], count[i] = lens[i] + 1, count[i] + 1


def test_captured_steps_replay():
    b = Batch([0] * 4, [100, 700, 300, 1], 2, 2, 128, 16, g4=True, seed=1)
    kv, lens, pages, _, num = b.gpu()
    w, budgets = random_weights(b).cuda(), torch.full((len(b.kv_lens),), 80, dtype=torch.int32, device="cuda")
    start, w0 = entries(b, "grown").cuda(), w.clone()

    def call(cache, came):
        return api.rpa_evict_kv_cache(cache, lens, pages, num, w, budgets, 80, sinks=1, recent=5, weights_out=w, positions=came,
                                      slots_out=torch.zeros(len(b.kv_lens), 2, 80, dtype=torch.int32, device="cuda"))

    call(kv.clone(), start.clone())
    torch.cuda.synchronize()
    mine, came = kv.clone(), start.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(mine, came)
    for m in ([100, 700, 300, 1], [90, 81, 79, 1]):
        lens[:4] = torch.tensor(m, dtype=torch.int32).cuda()
        for x, y in ((mine, kv), (came, start), (w, w0)):
            x.copy_(y)
        graph.replay()
        got_w = w.clone()
        w.copy_(w0)
        other, other_came = kv.clone(), start.clone()
        want = call(other, other_came)
        assert all(torch.equal(x, y) for x, y in zip(out, want)) and torch.equal(mine, other)
        assert torch.equal(came, other_came) and torch.equal(got_w, w)


def test_positions_are_checked():
    b = Batch([0] * 2, [30, 40], 2, 2, 128, 16)
    kv, lens, pages, _, num = b.gpu()
    w, bud = random_weights(b).cuda(), torch.full((3,), 8, dtype=torch.int32, device="cuda")
    came = torch.full(w.shape, -1, dtype=torch.int32, device="cuda")
    for bad in (came.float(), came.long(), came[:-1], came.transpose(1, 2), came.cpu()):
        with pytest.raises(ValueError):
            api.rpa_evict_kv_cache(kv, lens, pages, num, w, bud, 8, positions=bad)
    with pytest.raises(api.RpaError):
        api.rpa_evict_kv_cache(kv, lens, pages, num, w, bud, 8, positions=w.view(torch.int32))
    assert row_bytes(128) == kv.shape[-1]
