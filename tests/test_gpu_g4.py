"""The 4-bit cache on the GPU: what the update writes, what the read gives back and the attention over it, against their
float64 forms."""
import math

import pytest
import torch

import plain
from long_context import BF16, Batch, group_of, pack_rows, row_bytes, unpack_rows
from ragged_paged_attention_gb300 import api

pytestmark = pytest.mark.gpu

LENS = ([1, 3, 0, 2, 40, 1, 300, 17, 5], [1, 700, 64, 2, 40, 1500, 1300, 17, 2000])


def rows_of(t, hq, hkv, d, strided, seed=0):
    g = torch.Generator().manual_seed(seed)
    if strided:
        x = torch.randn(t, (hq + 2 * hkv) * d, generator=g).to(BF16)
        return tuple(x[:, a * d:(a + h) * d].unflatten(1, (h, d)) for a, h in ((0, hq), (hq, hkv), (hq + hkv, hkv)))
    return tuple(torch.randn(t, h, d, generator=g).to(BF16) for h in (hq, hkv, hkv))


def on_gpu(x):
    """x on the GPU with its strides."""
    return torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda").copy_(x)


def update(b, q, k, v, table, **kw):
    """(kv, q_out, error bits) of the call into a copy of the batch's cache."""
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    kv, lens, pages, cu, num = b.gpu()
    out = torch.full(q.shape, 7.0, dtype=BF16, device="cuda")
    got, back = api.rpa_g4_update_kv_cache(on_gpu(q), on_gpu(k), on_gpu(v), kv, lens, pages, cu, num, table, q_out=out,
                                           workspace=ws, **kw)
    assert got is out and back is kv
    return kv, out, api.check_device_status(ws)


def slots_of(b):
    """Each token's slot and position."""
    at = [p[k - n:] for p, n, k in zip(b.place, b.q_lens, b.lens)]
    return torch.cat(at), torch.cat([torch.arange(k - n, k) for n, k in zip(b.q_lens, b.lens)])


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("hq,hkv,d,ps", [(4, 4, 64, 16), (8, 2, 128, 16), (4, 2, 256, 32), (6, 1, 128, 12), (3, 3, 64, 1)])
def test_update_without_a_turn_writes_the_definitions_bytes(hq, hkv, d, ps, strided):
    b = Batch(*LENS, hq, hkv, d, ps, seed=d + ps)
    q, k, v = rows_of(b.t + 2, hq, hkv, d, strided)
    kv, out, bits = update(b, q, k, v, api.make_rope_table(0))
    assert bits == 0
    want = b.kv.clone()
    slot, _ = slots_of(b)
    want.flatten(0, 1)[slot] = pack_rows(k[:b.t], v[:b.t])
    got = kv.cpu()
    n = d // group_of(d)  # zeros of either sign are one value
    for x in (got, want):
        p = x[..., d:].contiguous().view(BF16)
        x[..., d:] = torch.where(p == 0, torch.zeros_like(p), p).view(torch.uint8)
        assert p.shape[-1] == 4 * n
    assert torch.equal(got, want)
    assert torch.equal(out[:b.t].cpu(), q[:b.t]) and (out[b.t:].float() == 7.0).all()


@pytest.mark.parametrize("d,rot,inter", [(64, 64, False), (64, 32, True), (128, 128, False), (128, 128, True), (128, 64, False),
                                         (128, 48, True), (256, 256, False), (256, 128, False), (256, 16, True)])
def test_update_turns_then_rounds(d, rot, inter):
    hq, hkv, ps = 4, 2, 16
    b = Batch(*LENS, hq, hkv, d, ps, seed=rot)
    q, k, v = rows_of(b.t + 2, hq, hkv, d, True, seed=1)
    kv, out, bits = update(b, q, k, v, api.make_rope_table(rot, interleaved=inter))
    assert bits == 0
    slot, pos = slots_of(b)
    freq, amp = plain.frequencies(rot)
    turned, slack = plain.rope(k[:b.t], pos, freq, amp, inter), plain.rope_slack(k[:b.t], freq, amp, inter)
    got = kv.cpu()
    rows = got.flatten(0, 1)[slot]
    gk, gv = unpack_rows(rows, d)
    # a value is rounded to bf16, then to the nearest of 16 steps s apart (the greatest may lie 15 * 2^-8 s beyond the
    # last, which is less than s / 2): half a step and the rounding off the turned value. s itself is 2^-8 of itself off a
    # 15th of the range of the rounded values, each bound above
    off = turned.abs() * 2.0 ** -8 + slack
    span = turned.unflatten(-1, (-1, group_of(d)))
    s = (span.amax(-1) - span.amin(-1) + 2 * off.unflatten(-1, (-1, group_of(d))).amax(-1)) / 15 * (1 + 2.0 ** -8)
    assert ((gk - turned).abs() <= s.repeat_interleave(group_of(d), -1) / 2 * (1 + 2.0 ** -20) + off).all()
    assert torch.equal(gv, unpack_rows(pack_rows(k[:b.t], v[:b.t]), d)[1])
    want_q = plain.rope(q[:b.t], pos, freq, amp, inter)
    assert ((out[:b.t].cpu().double() - want_q).abs() <= plain.half_step(want_q, BF16) * (1 + 2.0 ** -8) + plain.rope_slack(q[:b.t], freq, amp, inter) * 1.01).all()
    other = torch.ones(b.total * ps, dtype=torch.bool)
    other[slot] = False
    assert torch.equal(got.flatten(0, 1)[other], b.kv.flatten(0, 1)[other])


def test_update_of_odd_values():
    d, hkv = 128, 2
    b = Batch([6], [6], 2, hkv, d, 16)
    q, k, v = rows_of(8, 2, hkv, d, False)
    k[0], v[0] = 0.0, 3.5                      # one value: no step
    k[1, 0, 3], v[1, 1, 70] = math.inf, -math.inf
    k[2, 0, 5], v[2, 0, 0] = math.nan, math.nan
    k[3] = k[3] * 2.0 ** 100                   # beyond what is held
    v[3] = v[3] * 2.0 ** -130                  # subnormals
    k[4] = torch.arange(d).float().mul(0.5).to(BF16)  # quotients in the middle between two numbers
    v[4] = torch.arange(d).float().sub(64).to(BF16)
    kv, _, bits = update(b, q, k, v, api.make_rope_table(0))
    assert bits == 0
    slot, _ = slots_of(b)
    got, want = kv.cpu().flatten(0, 1)[slot], pack_rows(k[:6], v[:6])
    for x, y in zip(unpack_rows(got, d), unpack_rows(want, d)):
        assert torch.equal(x, y) and x.isfinite().all()


@pytest.mark.parametrize("hkv,d,ps", [(4, 64, 16), (2, 128, 12), (8, 128, 16), (2, 256, 32), (1, 64, 1)])
def test_read_gives_the_values_of_the_batchs_tokens(hkv, d, ps):
    b = Batch(*LENS, hkv, hkv, d, ps, seed=3)
    kv, lens, pages, cu, num = b.gpu()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    k, v = (torch.full((b.t + 3, hkv, d), 7.0, dtype=BF16, device="cuda") for _ in range(2))
    got = api.rpa_g4_read_kv_cache(kv, lens, pages, cu, num, k_out=k, v_out=v, workspace=ws)
    assert got[0] is k and got[1] is v and api.check_device_status(ws) == 0
    slot, _ = slots_of(b)
    for x, y in zip((k, v), unpack_rows(b.kv.flatten(0, 1)[slot], d)):
        assert torch.equal(x[:b.t].cpu(), y.float().to(BF16)) and (x[b.t:].float() == 7.0).all()
    # every key of the sequences
    whole = torch.cat([torch.zeros(1, dtype=torch.int32), lens.cpu()[:len(b.lens)].cumsum(0).int(), torch.full((1,), 10 ** 9).int()])
    k, v = api.rpa_g4_read_kv_cache(kv, lens, pages, whole.cuda(), num, sum(b.lens))
    for i, x in enumerate((k, v)):
        assert torch.equal(x.cpu(), torch.cat([b.values(j)[i] for j in range(len(b.lens))]).float().to(BF16))


def attend(b, **kw):
    kv, lens, pages, cu, num = b.gpu()
    q = b.q.cuda()
    ws = torch.zeros(api.rpa_g4_workspace_size(api.make_g4_params(q, kv, pages)), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 7.0)
    assert api.rpa_g4_forward(q, kv, lens, pages, cu, num, out=out, workspace=ws, **kw) is out
    return out, api.check_device_status(ws)


def check(b, **kw):
    kw.setdefault("sm_scale", b.d ** -0.5)
    out, bits = attend(b, **kw)
    assert bits == 0, hex(bits)
    want = b.attention(kw["sm_scale"], kw.get("sliding_window"), kw.get("soft_cap"))
    got = out[:b.t].double().cpu()
    assert (out[b.t:].float() == 7.0).all()
    assert not got.isnan().any()
    if not b.t:
        return out
    # Roundings of 2^-8 at most, 2^-8 / sqrt(3) in the root mean square, that are independent: of the output, of P (or
    # P s) and, for long queries, of V, each of the values' size where a row sees few keys (outputs of long averages
    # are smaller, and so are the errors); and of K, which moves a score by sm_scale sqrt(sum (q k 2^-8)^2 / 3), for
    # unit q and k sm_scale sqrt(d) 2^-8 / sqrt(3), and a weight by that share of itself
    rel = (got - want).norm() / want.norm()
    tol = 2.0 ** -8 / math.sqrt(3) * math.sqrt(3 + kw["sm_scale"] ** 2 * b.d)
    assert rel <= tol, (rel, tol)
    # the largest of up to 2^21 such errors lies within 6 of their deviations, on values of up to about 4.5
    assert (got - want).abs().max() <= 6 * tol * max(1.0, float(want.abs().max()))
    return out


@pytest.mark.parametrize("hq,hkv,d,ps", [(4, 4, 64, 16), (8, 2, 128, 16), (4, 2, 256, 32), (6, 1, 128, 8), (3, 3, 64, 64),
                                         (8, 8, 128, 4), (5, 1, 64, 12), (16, 1, 128, 128), (2, 1, 256, 1), (24, 2, 256, 16)])
def test_ragged_lengths(hq, hkv, d, ps):
    check(Batch(*LENS, hq, hkv, d, ps, seed=hq * d + ps))


@pytest.mark.parametrize("hq,hkv,ps", [(16, 8, 32), (8, 4, 16), (8, 4, 12), (24, 12, 1), (32, 4, 64), (6, 6, 16)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_numbers_of_kv_heads(hq, hkv, ps, d):
    check(Batch(*LENS, hq, hkv, d, ps, seed=hq * d + ps))
    check(Batch([1, 2, 1], [5000, 3, 900], hq, hkv, d, ps, seed=hkv), sliding_window=700)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_lens,kv_lens", [([1] * 40, list(range(1, 3000, 75))), ([1], [20000]), ([1, 1], [1, 2]), ([1], [16]), ([4], [17]),
                                            ([129], [129]), ([64, 64], [127, 129]), ([1000], [1000]), ([0, 0], [5, 0]),
                                            ([256, 1], [257, 4000])])
def test_batch_shapes(q_lens, kv_lens, d):
    check(Batch(q_lens, kv_lens, 8, 2, d, 16, seed=len(q_lens)))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window,cap", [(1, None), (17, None), (300, None), (None, 5.0), (200, 30.0), (5000, 2.0)])
def test_window_and_soft_cap(window, cap, d):
    check(Batch(*LENS, 8, 2, d, 16, seed=d), sliding_window=window, soft_cap=cap)


@pytest.mark.parametrize("scale", [-0.125, -1.5, 0.0, 1e-30])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_scales_of_either_sign(scale, d):
    check(Batch(*LENS, 4, 2, d, 16, seed=d), sm_scale=scale)


@pytest.mark.parametrize("hq,hkv", [(12, 2), (40, 5), (48, 1), (71, 1), (128, 1), (160, 1), (16, 16)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_group_sizes(hq, hkv, d):
    check(Batch([1, 3, 0, 2, 40, 1, 30], [1, 700, 64, 2, 40, 600, 130], hq, hkv, d, 16, seed=hq))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("up", [2.0 ** -20, 1.0, 2.0 ** 20])
def test_scales_of_the_values(up, d):
    # queries and keys whose sizes cancel, values far from one; outputs go with V's size
    b = Batch(*LENS, 8, 2, d, 16, seed=d)
    one = check(b)
    n = d // group_of(d)
    p = b.kv[..., d:].contiguous().view(BF16).unflatten(-1, (2, 2 * n))
    p[..., 0, :] *= up
    p[..., 1, :] *= 2.0 ** 30
    b.kv[..., d:] = p.flatten(-2).view(torch.uint8)
    b.q = (b.q.float() / up).to(BF16)
    got, bits = attend(b, sm_scale=d ** -0.5)
    assert bits == 0
    # Powers of two change no rounding of the keys. V at its own size and P with it are f16 in long queries (2^-11), past
    # f16's range bf16: P, V and both outputs then have independent roundings of 2^-8 at most, 2^-8 / sqrt(3) in the
    # root mean square
    a, c = one[:b.t].double(), got[:b.t].double() / 2.0 ** 30
    assert (a - c).norm() <= 2 * 2.0 ** -8 / math.sqrt(3) * a.norm()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("up", [2.0 ** -5, 0.25, 4.0])
def test_sizes_of_v_within_f16(up, d):
    b = Batch(*LENS, 8, 2, d, 16, seed=d)
    one = check(b)
    n = d // group_of(d)
    p = b.kv[..., d:].contiguous().view(BF16).unflatten(-1, (2, 2 * n))
    p[..., 1, :] *= up
    b.kv[..., d:] = p.flatten(-2).view(torch.uint8)
    got = check(b)
    # powers of two change no rounding; the pieces of a sequence join in another order, which float32 sums show
    a, c = one[:b.t].double(), got[:b.t].double() / up
    assert (a - c).norm() <= 1e-3 * a.norm()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_key_of_nearly_all_the_weight(d):
    # the first key takes all but some 2^-12 of each row and has no value: what is left is the others' average
    b = Batch([300, 40], [900, 400], 4, 2, d, 16, seed=d)
    n = d // group_of(d)
    p = b.kv[..., d:].contiguous().view(BF16).unflatten(-1, (2, 2 * n))
    for i in range(2):
        p[int(b.table[i, 0]), 0, :, 0, 0::2] = 0.0         # a key of ones, no values
        p[int(b.table[i, 0]), 0, :, 0, 1::2] = 1.0
        p[int(b.table[i, 0]), 0, :, 1] = 0.0
    b.kv[..., d:] = p.flatten(-2).view(torch.uint8)
    scale = d ** -0.5
    # the queries' sums put the first key's scores log(900 * 2^12) above zero
    b.q = (b.q.float() + math.log(900 * 2.0 ** 12) / (scale * d)).to(BF16)
    got, bits = attend(b, sm_scale=scale)
    assert bits == 0
    want = b.attention(scale)
    # check's roundings (queries of a greater size); weights of 2^-22 of the greatest, held in f16 times 2^7 in steps of 2^-24,
    # keep 2^-10 of themselves, beside which the 2^-8 leave that out
    norm_q = float((b.q[:b.t].double().pow(2).sum(-1) / d).sqrt().mean())
    tol = 6 * 2.0 ** -8 / math.sqrt(3) * math.sqrt(3 + norm_q ** 2)
    err, size = (got[:b.t].double().cpu() - want).norm(dim=-1), want.norm(dim=-1)
    assert (size > 0).all() and (err <= tol * size).all(), float((err / size).max())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("run", [64, 13])
def test_sizes_of_v_from_key_to_key(run, d):
    # V of runs of keys at sizes within f16's range, above and below it, and zeros; a row sees the nearest 20 keys, or all
    b = Batch([300, 1, 90], [700, 500, 90], 4, 2, d, 16, seed=d)
    n = d // group_of(d)
    sizes = torch.tensor([1.0, 2.0 ** 20, 2.0 ** -14, 0.0, 0.125, 2.0 ** 40, 2.0 ** -30])
    p = b.kv[..., d:].contiguous().view(BF16).unflatten(-1, (2, 2 * n))
    for i, kv_len in enumerate([700, 500, 90]):
        key = torch.arange(kv_len)
        page = b.table[i, key // 16].long()
        p[page, key % 16, :, 1, :] *= sizes[key // run % len(sizes)].to(BF16)[:, None, None]
    b.kv[..., d:] = p.flatten(-2).view(torch.uint8)
    for window in (20, None):
        got, bits = attend(b, sm_scale=d ** -0.5, sliding_window=window)
        assert bits == 0
        want = b.attention(d ** -0.5, window)
        # each row by itself, within 6 deviations of check's roundings
        tol = 6 * 2.0 ** -8 / math.sqrt(3) * math.sqrt(3 + 1)
        err, size = (got[:b.t].double().cpu() - want).norm(dim=-1), want.norm(dim=-1)
        assert (err <= tol * size).all(), float((err / size.clamp_min(1e-300)).max())


def test_long_context_offsets_past_32_bits():
    # 1.9 M slots of 8 heads: rows beyond 2 GB, the sequence's pages at the far end
    hkv, d, ps = 8, 128, 16
    pages = 2 ** 31 // (ps * hkv * row_bytes(d)) + 200
    b = Batch([1, 40], [900, 600], 8, hkv, d, ps, seed=5)
    kv = torch.zeros(pages, ps, hkv, row_bytes(d), dtype=torch.uint8, device="cuda")
    kv[pages - b.total:] = b.kv.cuda()
    table = torch.where(b.table < 2 ** 30, b.table + (pages - b.total), b.table).cuda()
    _, lens, _, cu, num = b.gpu()
    got = api.rpa_g4_forward(b.q.cuda(), kv, lens, table, cu, num, sm_scale=d ** -0.5)[:b.t].double().cpu()
    want = b.attention(d ** -0.5)
    assert (got - want).norm() <= 5e-3 * want.norm()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_sequences(d):
    g = torch.Generator().manual_seed(5)
    q_lens = torch.randint(0, 3, (2500,), generator=g)
    kv_lens = q_lens + torch.randint(0, 40, (2500,), generator=g)
    check(Batch(q_lens.tolist(), kv_lens.tolist(), 4, 2, d, 16, seed=6))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_pages_shared_by_sequences(d):
    b = Batch([1, 30, 2, 64], [1200, 600, 700, 1100], 8, 2, d, 16, seed=6)
    for i in range(1, 4):
        b.table[i] = b.table[0]
        b.place[i] = b.place[0][:b.lens[i]]
    check(b)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_keys_that_no_row_sees_may_hold_anything(d):
    # a window leaves a sequence's first keys out: NaN and infinite scales there change nothing
    b = Batch([1, 2, 50, 300], [700, 333, 400, 900], 8, 2, d, 16, seed=1)
    want, bits = attend(b, sm_scale=0.1, sliding_window=100)
    for i, k in enumerate(b.lens):
        gone = k - b.q_lens[i] - 100 + 1
        rows = b.kv.flatten(0, 1)
        rows[b.place[i][:gone], :, d:] = torch.tensor([255, 255, 128, 127], dtype=torch.uint8).repeat(2 * d // group_of(d))
    got, bits2 = attend(b, sm_scale=0.1, sliding_window=100)
    assert bits == bits2 == 0 and torch.equal(got[:b.t].view(torch.int16), want[:b.t].view(torch.int16))


@pytest.mark.parametrize("kind,q_lens", [(api.BATCH_DECODE_ONLY, [1, 2, 0, 4]), (api.BATCH_PREFILL_ONLY, [40, 5, 0, 300])])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_batch_kinds(kind, q_lens, d):
    b = Batch(q_lens, [700, 64, 9, 1000], 8, 2, d, 16, seed=2)
    check(b, batch_kind=kind)
    b.q_lens[0] = 5 if kind == api.BATCH_DECODE_ONLY else 1  # (a sequence of the other class is left out)
    b.cu[1:5] = torch.tensor(b.q_lens, dtype=torch.int32).cumsum(0)
    b.q = torch.cat([b.q[:1]] * (sum(b.q_lens) + 2))
    out, bits = attend(b, sm_scale=0.1, batch_kind=kind)
    assert bits == 0x80 and (out[:b.q_lens[0]].float() == 7.0).all()


def test_bad_metadata_is_recorded_and_skipped():
    for d in (64, 128, 256):
        for change, bit in (("page", 0x08), ("q", 0x02), ("kv", 0x04), ("tokens", 0x10), ("num", 0x01)):
            b = Batch([1, 20, 1], [300, 500, 40], 8, 2, d, 16, seed=3)
            if change == "page":
                b.table[1, 3] = b.total
            elif change == "q":
                b.kv_lens[1] = 19
            elif change == "kv":
                b.kv_lens[1] = b.table.shape[1] * 16 + 1
            elif change == "tokens":
                b.cu[2:4] = torch.tensor([10 ** 6, 10 ** 6 + 1])
            else:
                b.num[0] = 9
            out, bits = attend(b, sm_scale=0.1)
            assert bits & bit, (d, change, bits)
            if change in ("q", "kv"):
                assert (out[1:21].float() == 7.0).all() and not out[:1].isnan().any()
            if change == "num":
                assert (out.float() == 7.0).all()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_captured_call_replays_over_other_batches(d):
    b = Batch([1, 3, 40, 1], [100, 700, 300, 1], 8, 2, d, 16, seed=1, pad=200)
    kv, lens, pages, cu, num = b.gpu()
    q = b.q.nan_to_num(0.0).cuda()
    call = lambda: api.rpa_g4_forward(q, kv, lens, pages, cu, num, sm_scale=0.1)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for q_lens in ([1, 3, 40, 1], [1, 100, 0, 1], [60, 1, 1, 0]):
        cu[:5] = torch.tensor([0] + q_lens, dtype=torch.int32).cumsum(0).cuda()
        lens[:4] = torch.tensor([max(n, k) if n < 100 else 700 for n, k in zip(q_lens, (100, 700, 300, 1))], dtype=torch.int32).cuda()
        out.fill_(7.0)
        graph.replay()
        want = call()
        t = sum(q_lens)
        assert torch.equal(out[:t].view(torch.int16), want[:t].view(torch.int16))


def test_calls_on_two_streams():
    b = Batch(*LENS, 8, 2, 128, 16, seed=1)
    kv, lens, pages, cu, num = b.gpu()
    q = b.q.cuda()
    want = api.rpa_g4_forward(q, kv, lens, pages, cu, num, sm_scale=0.1)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(10):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(api.rpa_g4_forward(q, kv, lens, pages, cu, num, sm_scale=0.1))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[:b.t].view(torch.int16), want[:b.t].view(torch.int16))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_an_item_type_follows_from_its_own_values(d):
    # V of some heads and sequences beyond f16's range, others within it: each sequence's outputs are the same alone and among the
    # others, in every run, whichever order the SMs take the items in
    q_lens, kv_lens = [700, 40, 600, 90, 500], [900, 900, 600, 300, 1200]
    b = Batch(q_lens, kv_lens, 8, 4, d, 16, seed=d)
    n = d // group_of(d)
    p = b.kv[..., d:].contiguous().view(BF16).unflatten(-1, (2, 2 * n))
    for i in range(5):
        for h in range(4):
            if (i + h) % 2:
                at = b.place[i]
                p[at // 16, at % 16, h, 1] *= 2.0 ** (10 if h % 2 else -20)
    b.kv[..., d:] = p.flatten(-2).view(torch.uint8)
    first, bits = attend(b, sm_scale=d ** -0.5)
    assert bits == 0
    want = b.attention(d ** -0.5)
    tol = 6 * 2.0 ** -8 / math.sqrt(3) * math.sqrt(3 + 1)
    err, size = (first[:b.t].double().cpu() - want).norm(dim=-1), want.norm(dim=-1)
    assert (err <= tol * size).all(), float((err / size).max())
    for _ in range(5):
        got, bits = attend(b, sm_scale=d ** -0.5)
        assert bits == 0 and torch.equal(got[:b.t].view(torch.int16), first[:b.t].view(torch.int16))
    kv, lens, pages, _, num = b.gpu()
    q = b.q.cuda()
    num.fill_(1)
    for i, m in enumerate(q_lens):
        a = int(b.cu[i])
        cu = torch.tensor([0, m], dtype=torch.int32, device="cuda")
        got = api.rpa_g4_forward(q[a:a + m], kv, lens[i:i + 1], pages[i:i + 1].contiguous(), cu, num, sm_scale=d ** -0.5)
        assert torch.equal(got.view(torch.int16), first[a:a + m].view(torch.int16))
