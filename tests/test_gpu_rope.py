"""GPU parity of rope_apply and rpa_rope_update_kv_cache against their float64 forms."""
import math

import numpy as np
import pytest
import torch

import plain
from ragged_paged_attention_gb300 import api

pytestmark = pytest.mark.gpu

LLAMA3 = {"type": "llama3", "factor": 8.0, "low_freq_factor": 1.0, "high_freq_factor": 4.0,
          "original_max_position": 8192}
YARN = {"type": "yarn", "factor": 40.0, "original_max_position": 4096}
BF16, FP8, INT8, INT4 = torch.bfloat16, torch.float8_e4m3fn, torch.int8, torch.uint8


def randn(seed, *shape, dtype=BF16):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape, dtype=np.float32)).to(dtype)


def bits(x):
    return x.contiguous().view(torch.int16 if x.element_size() == 2 else torch.uint8)


def rows(x, at):
    """x[at] of rows [n, heads, elements] (an e4m3 tensor on the CPU has no indexing of its own)."""
    return x.view(torch.uint8)[at].view(x.dtype) if x.element_size() == 1 else x[at]


def near(got, ref, slack):
    """got (bf16) is ref rounded once, up to the arithmetic's slack."""
    d = (got.double() - ref).abs()
    assert not d.isnan().any()
    over = d - plain.half_step(ref.abs() + slack, BF16) - slack
    assert (over <= 0).all(), over.max().item()


POSITIONS = [0, 1, -1, 7, 4095, 131071, 1 << 20, -(1 << 20), 2**31 - 1, -2**31]


@pytest.mark.parametrize("T,hq,hk,d,rot,inter,scaling", [
    (1, 1, 0, 64, 64, False, None), (10, 4, 2, 64, 64, True, YARN), (10, 32, 8, 128, 128, False, LLAMA3),
    (37, 16, 8, 256, 256, True, None), (10, 3, 1, 96, 24, False, None), (10, 3, 1, 96, 96, False, LLAMA3),
    (10, 5, 5, 80, 20, False, None), (11, 7, 1, 80, 10, True, None), (11, 2, 1, 32, 6, False, None),
    (10, 2, 2, 512, 256, False, None), (9, 2, 2, 512, 64, True, None), (5, 9, 1, 16, 16, False, None),
    (5, 9, 1, 16, 2, False, None), (10, 2, 1, 128, 0, False, None), (700, 6, 2, 192, 64, False, YARN),
    (3001, 4, 1, 128, 128, True, LLAMA3)])
def test_apply(T, hq, hk, d, rot, inter, scaling):
    q, k = randn(1, T, hq, d), randn(2, T, hk, d) if hk else None
    pos = torch.tensor((POSITIONS * (T // len(POSITIONS) + 1))[:T], dtype=torch.int32)
    t = api.make_rope_table(rot, base=500000.0, interleaved=inter, scaling=scaling)
    f, amp = plain.frequencies(rot, 500000.0, scaling)
    for inverse in (False, True):
        qo, ko = api.rope_apply(q.cuda(), k.cuda() if hk else None, pos.cuda(), t, inverse=inverse)
        assert (ko is None) == (hk == 0)
        for x, y in ((q, qo), (k, ko)) if hk else ((q, qo),):
            # at |position| 2^31 the table's own steps (float64 frequencies, relative 2^-52, and 2^-64
            # turns) move the angle by up to 2^31 * (f 2^-51 + 2 pi 2^-64) < 2^-19
            far = (pos.double().abs()[:, None, None] * 2.0 ** -50) * (x.double().abs().amax(-1, keepdim=True) * 2 * amp)
            near(y.cpu(), plain.rope(x, pos, f, amp, inter, inverse), plain.rope_slack(x, f, amp, inter) + far)


def test_apply_strides_layouts_and_in_place():
    t, d = api.make_rope_table(64, interleaved=True), 64
    f, amp = plain.frequencies(64)
    pos = torch.arange(50, 69, dtype=torch.int32)
    ref = lambda x: plain.rope(x, pos, f, amp, True)  # noqa: E731
    slack = lambda x: plain.rope_slack(x, f, amp, True)  # noqa: E731
    # the last 64 of each head's 192 elements, out dense; the other elements stay as they are
    x = randn(3, 19, 5, 192)
    g = x.cuda()
    out, _ = api.rope_apply(g[..., 128:], None, pos.cuda(), t)
    assert out.is_contiguous()
    near(out.cpu(), ref(x[..., 128:]), slack(x[..., 128:]))
    # the same in place
    api.rope_apply(g[..., 128:], None, pos.cuda(), t, q_out=g[..., 128:])
    assert torch.equal(bits(g[..., 128:].cpu()), bits(out.cpu()))
    assert torch.equal(bits(g[..., :128].cpu()), bits(x[..., :128]))
    # q and k as slices of one projection's rows, in place; v stays
    x = randn(4, 19, 9 * d)
    g = x.cuda()
    cut = lambda y: (y[:, :5 * d].unflatten(1, (5, d)), y[:, 5 * d:7 * d].unflatten(1, (2, d)))  # noqa: E731
    api.rope_apply(*cut(g), pos.cuda(), t, q_out=cut(g)[0], k_out=cut(g)[1])
    for a, b in zip(cut(g.cpu()), cut(x)):
        near(a, ref(b), slack(b))
    assert torch.equal(bits(g[:, 7 * d:].cpu()), bits(x[:, 7 * d:]))
    # heads outside tokens, in and out
    x = randn(5, 5, 19, d)
    g = x.cuda().transpose(0, 1)
    out = torch.zeros(5, 19, d, dtype=BF16, device="cuda").transpose(0, 1)
    api.rope_apply(g, None, pos.cuda(), t, q_out=out)
    near(out.cpu(), ref(x.transpose(0, 1)), slack(x.transpose(0, 1)))
    # one token, one head: any stride of the dimensions of one entry
    one = randn(6, 3, 3, 72).cuda()[1:2, 2:3, 8:]
    near(api.rope_apply(one, None, pos[:1].cuda(), t)[0].cpu(), plain.rope(one.cpu(), pos[:1], f, amp, True),
         plain.rope_slack(one.cpu(), f, amp, True))


def test_apply_refusals_of_the_binding():
    t, pos = api.make_rope_table(64), torch.zeros(4, dtype=torch.int32, device="cuda")
    x = torch.zeros(4, 2, 64, dtype=BF16, device="cuda")
    for bad in (x.float(), x[:, 0], x.transpose(1, 2), torch.zeros(4, 2, 68, dtype=BF16, device="cuda")[..., :64],
                x[:, :1].expand(4, 3, 64), x.half()):
        with pytest.raises(ValueError):
            api.rope_apply(bad, None, pos, t)
    for kw in (dict(positions=pos[:3]), dict(positions=pos.long()), dict(positions=pos.cpu()), dict(k=x[:3]),
               dict(k=x[..., :32]), dict(q_out=x[:, :1]), dict(k_out=x)):
        args = {**dict(q=x, k=None, positions=pos, table=t), **kw}
        with pytest.raises(ValueError):
            api.rope_apply(**args)
    y = torch.zeros(8, 2, 64, dtype=BF16, device="cuda")
    with pytest.raises(api.RpaError):
        api.rope_apply(y[:4], None, pos, t, q_out=y[2:6])  # overlaps without being it
    q, k = api.rope_apply(x[:0], x[:0], pos[:0], t)
    assert q.shape == k.shape == (0, 2, 64)


def test_inverse_undoes_and_is_the_gradient():
    f, amp = plain.frequencies(32, 10000.0, YARN)
    t = api.make_rope_table(32, scaling=YARN)
    pos = torch.tensor([3, 50000, -9], dtype=torch.int32)
    x, g = randn(7, 3, 4, 64), randn(8, 3, 4, 64)
    y, _ = api.rope_apply(x.cuda(), None, pos.cuda(), t)
    # undone up to the amplitude's square on the turned elements and two roundings to bf16
    back, _ = api.rope_apply(y, None, pos.cuda(), t, inverse=True)
    scale = torch.ones(64, dtype=torch.float64)
    scale[:32] = amp * amp
    biggest = x.double().abs().amax() * amp * amp * 2
    assert (back.cpu().double() - x.double() * scale).abs().max() <= biggest * (2.0 ** -8 * 2 + 2.0 ** -20)
    # the gradient of sum(g * rope(x)): against the formula's (autograd in float64) and differences
    xd = x.double().requires_grad_()
    (plain.rope(xd, pos, f, amp, False) * g.double()).sum().backward()
    got, _ = api.rope_apply(g.cuda(), None, pos.cuda(), t, inverse=True)
    near(got.cpu(), xd.grad, plain.rope_slack(g, f, amp, False))
    for at in ((0, 1, 3), (1, 2, 40), (2, 0, 20), (1, 3, 31)):
        step = torch.zeros_like(xd)
        step[at] = 0.5
        with torch.no_grad():  # the map is linear: the difference is exact up to float64
            diff = ((plain.rope(xd + step, pos, f, amp, False) - plain.rope(xd - step, pos, f, amp, False)) * g.double()).sum()
        assert abs(got[at].item() - diff.item()) <= 2.0 ** -8 * abs(diff.item()) + 2.0 ** -20 * 8


# ------------------------------------------------------------------ the cache write
def make_batch(q_lens, kv_lens, hq, hkv, d, ps, dtype, *, seed, pad=0, unused=1, strided=False):
    """CPU tensors of one batch: random pages, garbage behind the last sequence, a patterned cache."""
    rng = np.random.default_rng(seed)
    n, T = len(q_lens), sum(q_lens) + pad
    pps = max(1, max(-(-k // ps) for k in kv_lens)) + 1
    total = sum(-(-k // ps) for k in kv_lens) + 2
    table = np.full((n + unused, pps), 2**31 - 1, np.int32)
    perm, at = rng.permutation(total).astype(np.int32), 0
    for s, k in enumerate(kv_lens):
        m = -(-k // ps)
        table[s, :m] = perm[at:at + m]
        at += m
    kvl = np.full(n + unused, 10**9, np.int32)
    kvl[:n] = kv_lens
    cu = np.full(n + unused + 1, -7, np.int32)
    cu[:n + 1] = np.concatenate([[0], np.cumsum(q_lens)])
    raw = rng.integers(0, 256, size=total * ps * 2 * hkv * d * {BF16: 4, FP8: 2, INT8: 2, INT4: 1}[dtype] // 2, dtype=np.uint8)
    kv = torch.from_numpy(raw).view(dtype).reshape(total, ps, 2 * hkv, -1)
    if strided:
        x = randn(seed + 1, T, (hq + 2 * hkv) * d)
        q, k, v = (x[:, a * d:(a + h) * d].unflatten(1, (h, d)) for a, h in ((0, hq), (hq, hkv), (hq + hkv, hkv)))
    else:
        q, k, v = randn(seed + 1, T, hq, d), randn(seed + 2, T, hkv, d), randn(seed + 3, T, hkv, d)
    return dict(q=q, k=k, v=v, kv=kv, kv_lens=torch.from_numpy(kvl), pages=torch.from_numpy(table), cu=torch.from_numpy(cu),
                num=torch.tensor([n], dtype=torch.int32), q_lens=q_lens, lens=kv_lens, ps=ps)


def slots_of(b):
    pos = torch.cat([torch.arange(k - n, k) for n, k in zip(b["q_lens"], b["lens"])])
    seq = torch.cat([torch.full((n,), s) for s, n in enumerate(b["q_lens"])])
    return pos, b["pages"][seq, pos // b["ps"]].long() * b["ps"] + pos % b["ps"]


def write(b, table, with_q=True, positions=None, workspace=None, **kw):
    """Runs the call on the GPU on copies; (q_out, cache) on the CPU. Strided inputs keep their strides."""
    same = b["q"].data_ptr() != b["k"].data_ptr() and not b["q"].is_contiguous()
    if same:
        base = b["q"]._base.cuda()
        q, k, v = (torch.as_strided(base, x.shape, x.stride(), x.storage_offset()) for x in (b["q"], b["k"], b["v"]))
    else:
        q, k, v = b["q"].cuda(), b["k"].cuda(), b["v"].cuda()
    kv = b["kv"].clone().cuda()
    q_out = torch.full(b["q"].shape, 7.0, dtype=BF16, device="cuda") if with_q else None
    out, kv2 = api.rpa_rope_update_kv_cache(q if with_q else None, k, v, kv, b["kv_lens"].cuda(), b["pages"].cuda(),
                                            b["cu"].cuda(), b["num"].cuda(), table, q_out=q_out, workspace=workspace,
                                            positions=None if positions is None else positions.cuda(), **kw)
    assert out is q_out and kv2 is kv
    torch.cuda.synchronize()
    return (q_out.cpu() if with_q else None), kv.cpu()


def check_write(b, q_out, kv, f, amp, inter, positions=None, k_scale=None, v_scale=None, skip=()):
    pos, slot = slots_of(b)
    t = len(pos)
    keep = torch.ones(t, dtype=torch.bool)
    keep[list(skip)] = False
    turn = pos if positions is None else positions[:t]
    if q_out is not None:
        near(q_out[:t][keep], plain.rope(b["q"][:t], turn, f, amp, inter)[keep], plain.rope_slack(b["q"][:t], f, amp, inter)[keep])
        rest = torch.ones(len(q_out), dtype=torch.bool)
        rest[:t][keep] = False
        assert (q_out[rest].float() == 7.0).all()
    dtype = kv.dtype
    flat = kv.flatten(0, 1)
    untouched = torch.ones(len(flat), dtype=torch.bool)
    untouched[slot[keep]] = False
    assert torch.equal(bits(rows(flat, untouched)), bits(rows(b["kv"].flatten(0, 1), untouched)))
    for part, x, scale in ((0, b["k"][:t], k_scale), (1, b["v"][:t], v_scale)):
        ref, slack = (plain.rope(x, turn, f, amp, inter), plain.rope_slack(x, f, amp, inter)) if part == 0 else \
            (x.double(), torch.zeros(x.shape, dtype=torch.float64))
        s = scale or 1.0
        # the division is a product with the rounded reciprocal: two roundings of 2^-24
        ref, slack = ref / s, slack / abs(s) + (ref / s).abs() * 2.0 ** -22 * (scale is not None)
        if dtype in plain.LIMITS:
            ref = ref.clamp(*plain.LIMITS[dtype])
        got = plain.stored_values(rows(flat, slot))[:, part::2]
        over = ((got - ref).abs() - plain.half_step(ref.abs() + slack, dtype) - slack)[keep]
        assert (over <= 0).all(), (part, over.max().item())


@pytest.mark.parametrize("dtype,ks,vs", [(BF16, None, None), (BF16, 0.37, 1.7), (FP8, None, None), (FP8, 0.011, 0.02),
                                         (INT8, 0.02, 0.03), (INT4, 0.3, 0.4)], ids=str)
@pytest.mark.parametrize("hq,hkv,d,rot,inter,ps,strided", [
    (8, 2, 128, 128, False, 16, True), (6, 2, 64, 64, True, 8, False), (4, 4, 256, 64, False, 32, True),
    (3, 1, 96, 24, False, 4, False), (5, 5, 192, 192, True, 12, False), (2, 1, 128, 20, True, 16, True),
    (3, 3, 96, 96, False, 16, True), (4, 1, 128, 16, False, 1, False)])
def test_update(dtype, ks, vs, hq, hkv, d, rot, inter, ps, strided):
    b = make_batch([1, 0, 37, 1, 5], [40000, 70, 37, 1, 300], hq, hkv, d, ps, dtype, seed=d + rot, pad=3, strided=strided)
    t = api.make_rope_table(rot, base=500000.0, interleaved=inter, scaling=LLAMA3)
    f, amp = plain.frequencies(rot, 500000.0, LLAMA3)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    q_out, kv = write(b, t, k_scale=ks, v_scale=vs, workspace=ws)
    assert api.check_device_status(ws) == 0
    check_write(b, q_out, kv, f, amp, inter, k_scale=ks, v_scale=vs)


@pytest.mark.parametrize("rot", [6, 10, 66])
def test_update_odd_pair_counts(rot):
    for dtype in (BF16, FP8, INT8):
        b = make_batch([3, 20], [30, 20], 4, 2, 128, 16, dtype, seed=rot)
        t, (f, amp) = api.make_rope_table(rot), plain.frequencies(rot)
        check_write(b, *write(b, t, k_scale=0.05, v_scale=0.05), f, amp, False, k_scale=0.05, v_scale=0.05)


@pytest.mark.parametrize("n,T", [(1, 1), (1, 4000), (1500, 1), (300, 7)])
def test_update_batch_shapes(n, T):
    # one token; one long chunk; more sequences than a block looks through at once; several of each
    b = make_batch([T] * n, [T + (13 * s) % 90 for s in range(n)], 4, 2, 64, 16, BF16, seed=n, pad=1)
    t, (f, amp) = api.make_rope_table(64, scaling=YARN), plain.frequencies(64, 10000.0, YARN)
    check_write(b, *write(b, t), f, amp, False)


@pytest.mark.parametrize("n", [1022, 1023, 1024, 1100])
def test_update_of_many_sequences_with_empty_and_bad_ones(n):
    # either way of finding a token's sequence: lengths 0 to 2, one sequence whose kv_len is past its pages
    q_lens = [(3 * s + s // 7) % 3 for s in range(n)]
    b = make_batch(q_lens, [L + (5 * s) % 40 for s, L in enumerate(q_lens)], 4, 2, 64, 16, BF16, seed=n, pad=2)
    good = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in b.items()}
    bad = next(s for s in range(n // 2, n) if q_lens[s] == 2)
    b["kv_lens"][bad] = 10**6
    t, (f, amp) = api.make_rope_table(64), plain.frequencies(64)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    q_out, kv = write(b, t, workspace=ws)
    assert api.check_device_status(ws) == 0x04
    first = sum(q_lens[:bad])
    check_write(good, q_out, kv, f, amp, False, skip=range(first, first + 2))


def test_update_of_no_sequences():
    b = make_batch([2, 3], [20, 9], 4, 2, 128, 16, BF16, seed=1)
    b["num"][0] = 0
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    q_out, kv = write(b, api.make_rope_table(64), workspace=ws)
    assert (q_out.float() == 7.0).all() and torch.equal(bits(kv), bits(b["kv"])) and api.check_device_status(ws) == 0


def test_update_behind_four_gigabytes():
    # the last pages of a cache of 9.8 GB, with rows of another cache's size in front
    hq, hkv, d, ps, pages = 4, 4, 128, 16, 300000
    kv = torch.empty(pages, ps, 2 * hkv, d, dtype=BF16, device="cuda")
    kv[-3:].zero_()
    q, k, v = randn(1, 20, hq, d), randn(2, 20, hkv, d), randn(3, 20, hkv, d)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    t, (f, amp) = api.make_rope_table(128), plain.frequencies(128)
    api.rpa_rope_update_kv_cache(q.cuda(), k.cuda(), v.cuda(), kv, i32(20), table, i32(0, 20), i32(1), t)
    got = kv[[pages - 1, pages - 2]].flatten(0, 1)[:20].cpu()
    near(got[:, 0::2], plain.rope(k, torch.arange(20), f, amp, False), plain.rope_slack(k, f, amp, False))
    assert torch.equal(bits(got[:, 1::2]), bits(v))
    # and read from there: every query over the 20 keys
    out = api.rpa_cross_forward(q.cuda(), kv, i32(20), table, i32(0, 20), i32(1), sm_scale=0.1)
    ref = plain.attend_all(q, kv[-3:].cpu(), torch.tensor([20]), torch.tensor([[2, 1]]), torch.tensor([0, 20]), 1, sm_scale=0.1)
    assert (out.cpu().double() - ref).abs().max() <= 2e-2


def test_update_without_queries_other_positions_and_no_turn():
    b = make_batch([4, 1, 9], [4, 33, 100], 4, 2, 128, 16, FP8, seed=5, pad=2)
    t, (f, amp) = api.make_rope_table(128), plain.frequencies(128)
    pos = torch.tensor([5, -3, 1 << 20, 0, 9, 1, 2, 3, 4, 5, 6, 7, 8, 100000, 3, 3], dtype=torch.int32)
    q_out, kv = write(b, t, positions=pos, k_scale=0.02, v_scale=0.02)
    check_write(b, q_out, kv, f, amp, False, positions=pos, k_scale=0.02, v_scale=0.02)
    q_out, kv = write(b, t, with_q=False, k_scale=0.02, v_scale=0.02)
    assert q_out is None
    check_write(b, None, kv, f, amp, False, k_scale=0.02, v_scale=0.02)
    # nothing turns: a bf16 cache gets the bits of rpa_update_kv_cache
    b = make_batch([4, 1, 9], [4, 33, 100], 4, 2, 128, 16, BF16, seed=6)
    _, kv = write(b, api.make_rope_table(0), with_q=False)
    ref = b["kv"].clone().cuda()
    api.rpa_update_kv_cache(b["k"].cuda(), b["v"].cuda(), ref, b["kv_lens"].cuda(), b["pages"].cuda(), b["cu"].cuda(),
                            b["num"].cuda())
    assert torch.equal(bits(kv), bits(ref.cpu()))


@pytest.mark.parametrize("dtype", [BF16, FP8, INT8, INT4])
def test_update_of_extreme_values(dtype):
    # infinities, NaN and values past the type's range: saturated as documented, NaN kept or 0
    b = make_batch([2], [2], 2, 1, 64, 16, dtype, seed=9)
    v = torch.tensor([math.inf, -math.inf, math.nan, 3e38, -3e38, 449.0, -1000.0, 0.0], dtype=BF16)
    b["v"][:] = v.repeat(8)
    b["k"][:, :, 32:] = v.repeat(4)  # past rotary_dim: copied
    _, kv = write(b, api.make_rope_table(32))
    _, slot = slots_of(b)
    for part in (0, 1):
        got = plain.stored_values(rows(kv.flatten(0, 1), slot))[:, part, -8:]
        if dtype == BF16:
            assert torch.equal(got.nan_to_num(7.0, 1e39, -1e39), v.double().nan_to_num(7.0, 1e39, -1e39).expand_as(got))
            continue
        lo, hi = plain.LIMITS[dtype]
        want = v.double().clamp(lo, hi)
        want[2] = math.nan if dtype == FP8 else 0.0
        assert torch.equal(got.nan_to_num(1e9), want.nan_to_num(1e9).expand_as(got))


@pytest.mark.parametrize("what,code,skip", [
    ("page", 0x08, [0, 1, 2]), ("kv_len", 0x04, range(3, 8)), ("q_len", 0x02, range(3, 8)), ("tokens", 0x10, range(8, 10)),
    ("num", 0x01, range(10)), ("negative num", 0x01, range(10))])
def test_update_skips_bad_metadata(what, code, skip):
    b = make_batch([3, 5, 2], [20, 40, 2], 4, 2, 64, 16, BF16, seed=3, pad=1)
    good = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in b.items()}
    if what == "page":
        b["pages"][0, 1] = b["kv"].shape[0]  # positions 17-19 of sequence 0
    elif what == "kv_len":
        b["kv_lens"][1] = 10**6
    elif what == "q_len":
        b["kv_lens"][1] = 4
    elif what == "tokens":
        b["cu"][3] = 12  # past max_num_tokens
    else:
        b["num"][0] = 5 if what == "num" else -1
    t, (f, amp) = api.make_rope_table(64), plain.frequencies(64)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    q_out, kv = write(b, t, workspace=ws)
    assert api.check_device_status(ws) == code
    check_write(good, q_out, kv, f, amp, False, skip=skip)
    write(b, t)  # without a workspace nothing is recorded and nothing else changes


def test_update_refusals_of_the_binding():
    b = make_batch([3], [20], 4, 2, 64, 16, BF16, seed=3)
    t = api.make_rope_table(64)
    g = {k: v.cuda() for k, v in b.items() if isinstance(v, torch.Tensor)}
    good = dict(q=g["q"], new_k=g["k"], new_v=g["v"], kv_pages=g["kv"], kv_lens=g["kv_lens"], page_indices=g["pages"],
                cu_q_lens=g["cu"], num_seqs=g["num"], table=t)
    for bad in (dict(q=g["q"][:2]), dict(q=g["q"].float()), dict(new_k=g["k"][..., :32]), dict(new_v=g["v"][:, :1]),
                dict(new_v=g["v"][:2]), dict(kv_lens=g["kv_lens"][:1]), dict(cu_q_lens=g["cu"].long()), dict(num_seqs=g["num"].cpu()),
                dict(q=None, q_out=g["q"]), dict(q_out=g["q"][:, :2]), dict(positions=g["kv_lens"]), dict(table=None),
                dict(kv_pages=g["kv"].transpose(0, 1)), dict(new_k=g["k"].float())):
        with pytest.raises(ValueError):
            api.rpa_rope_update_kv_cache(**{**good, **bad})
    with pytest.raises(api.RpaError):
        api.rpa_rope_update_kv_cache(**{**good, "table": api.make_rope_table(128)})
    q, kv = api.rpa_rope_update_kv_cache(**{**good, "q": g["q"][:0], "new_k": g["k"][:0], "new_v": g["v"][:0]})
    assert q.shape[0] == 0 and kv is g["kv"]


def test_update_in_place_queries_on_another_stream():
    b = make_batch([3, 700], [20, 900], 8, 2, 128, 16, BF16, seed=4)
    t = api.make_rope_table(128, scaling=LLAMA3)
    want, cache = write(b, t)
    g = {k: v.cuda() for k, v in b.items() if isinstance(v, torch.Tensor)}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q, kv = api.rpa_rope_update_kv_cache(g["q"], g["k"], g["v"], g["kv"], g["kv_lens"], g["pages"], g["cu"], g["num"], t,
                                             q_out=g["q"])
    side.synchronize()
    assert torch.equal(bits(q.cpu()), bits(want)) and torch.equal(bits(kv.cpu()), bits(cache))
