"""GPU parity of rpa_cross_forward and rpa_rope_forward_update against their float64 forms, and the
operators together as a decoder layer uses them."""
import math

import numpy as np
import pytest
import torch

import oracle
import plain
from parity import TOL_BF16, TOL_FP8
from ragged_paged_attention_gb300 import api, workloads

pytestmark = pytest.mark.gpu

BF16, FP8, INT8, INT4 = torch.bfloat16, torch.float8_e4m3fn, torch.int8, torch.uint8


def batch(q_lens, kv_lens, hq, hkv, d, ps, *, dtype=BF16, seed=0, pad=2, **kw):
    """A ragged batch with every byte that must not be read poisoned (NaN slots past kv_len, page ids
    past the sequence, rows and metadata behind the last sequence)."""
    b = workloads.make_rpa(q_lens, kv_lens, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=ps, seed=seed,
                           kv_dtype=dtype, max_num_seqs=len(q_lens) + 1, max_num_tokens=max(1, sum(q_lens) + pad),
                           extra_pages=2, **kw)
    return b


def run(b, fill=7.0, workspace=True, **kw):
    g = b.to("cuda")
    opts = dict(sm_scale=b.sm_scale, soft_cap=b.soft_cap, k_scale=b.k_scale, v_scale=b.v_scale, **kw)
    ws = None
    if workspace:
        prm = api.make_rpa_params(g.q, g.kv_pages, g.page_indices, **opts)
        ws = torch.zeros(api.rpa_cross_workspace_size(prm), dtype=torch.uint8, device="cuda")
    out = torch.full_like(g.q, fill)
    got = api.rpa_cross_forward(g.q, g.kv_pages, g.kv_lens, g.page_indices, g.cu_q_lens, g.num_seqs, out=out, workspace=ws,
                                **opts)
    assert got is out
    torch.cuda.synchronize()
    return out.cpu(), 0 if ws is None else api.check_device_status(ws)


def reference(b):
    return plain.attend_all(b.q, b.kv_pages, b.kv_lens, b.page_indices, b.cu_q_lens, len(b.q_lens), sm_scale=b.sm_scale,
                            soft_cap=b.soft_cap, k_scale=b.k_scale, v_scale=b.v_scale)


def check(b, tol, **kw):
    out, bits = run(b, **kw)
    assert bits == 0, hex(bits)
    ref, t = reference(b), b.num_tokens
    err = (out[:t].double() - ref[:t]).abs()
    assert not err.isnan().any()
    assert err.max().item() <= tol if t else True, err.max().item()
    assert (out[t:].float() == 7.0).all()
    for s, k in enumerate(b.kv_lens_list):  # no key: exact zeros
        if k == 0:
            assert (out[int(b.cu_q_lens[s]):int(b.cu_q_lens[s + 1])] == 0).all()
    return out


# one key, fewer keys than queries and more, no keys, no queries, one token to several tiles
LENS = ([1, 3, 0, 2, 40, 1, 300, 17, 5], [1, 700, 64, 0, 9, 1500, 130, 0, 2000])


@pytest.mark.parametrize("hq,hkv,d,ps", [(4, 4, 64, 16), (8, 2, 128, 16), (4, 2, 256, 32), (6, 1, 128, 8), (3, 3, 64, 64),
                                         (8, 8, 128, 4), (5, 1, 64, 12), (4, 4, 96, 16), (2, 2, 192, 32), (16, 1, 128, 128)])
def test_ragged_lengths(hq, hkv, d, ps):
    check(batch(*LENS, hq, hkv, d, ps, seed=hq * d + ps), TOL_BF16)


@pytest.mark.parametrize("dtype,ks,vs", [(FP8, None, None), (FP8, 0.5, 2.0), (FP8, 0.37, 0.9), (INT8, 2.0**-6, 2.0**-6),
                                         (INT8, 0.013, 0.011), (INT4, 0.25, 0.3), (BF16, 0.7, 0.8)], ids=str)
@pytest.mark.parametrize("d,ps", [(64, 16), (128, 16), (256, 32), (128, 4)])
def test_cache_types(dtype, ks, vs, d, ps):
    b = batch(*LENS, 4, 2, d, ps, dtype=dtype, seed=d, k_scale=ks, v_scale=vs)
    # the accuracy target is absolute on outputs of unit-size values: it scales with V's largest
    unit = {FP8: 1.0, INT8: 64.0, INT4: 4.0, BF16: 1.0}[dtype] * (vs or 1.0)
    check(b, (TOL_BF16 if dtype == BF16 else TOL_FP8) * max(1.0, unit))


@pytest.mark.parametrize("cap", [2.0, 50.0])
def test_soft_cap(cap):
    check(batch(*LENS, 4, 2, 128, 16, seed=7, soft_cap=cap), TOL_BF16)


@pytest.mark.parametrize("q_lens,kv_lens", [([1] * 40, list(range(1, 3000, 75))), ([1], [20000]), ([1, 1], [0, 0]),
                                            ([600], [0]), ([600, 600], [0, 0]), ([129], [128]), ([4, 4], [127, 129]),
                                            ([2000], [3]), ([1], [1]), ([0, 0], [5, 0]), ([256, 1], [1, 4000])])
def test_batch_shapes(q_lens, kv_lens):
    check(batch(q_lens, kv_lens, 8, 2, 128, 16, seed=len(q_lens)), TOL_BF16)


@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, BF16), (128, FP8)])
def test_many_sequences(d, dtype):
    # more sequences than the plan's block has threads; a third without keys, some without queries
    rng = np.random.default_rng(5)
    q_lens = rng.integers(0, 3, 2500).tolist()
    kv_lens = (rng.integers(0, 40, 2500) * (rng.random(2500) < 0.7)).tolist()
    check(batch(q_lens, kv_lens, 4, 2, d, 16, dtype=dtype, seed=6), TOL_BF16 if dtype == BF16 else TOL_FP8)


@pytest.mark.parametrize("d", [64, 128])
def test_sequences_of_many_lengths_in_any_order(d):
    # more items than CTAs, in an order by length across more sequences than the plan's block has threads
    rng = np.random.default_rng(8)
    kv_lens = (rng.integers(0, 10, 1300) ** 3 * (rng.random(1300) < 0.9)).astype(int).tolist()
    q_lens = rng.integers(0, 4, 1300)
    q_lens[[7, 700, 1299]] = 300, 41, 33
    check(batch(q_lens.tolist(), kv_lens, 4, 2, d, 16, seed=9), TOL_BF16)


@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (8, 2, 64), (8, 2, 128), (2, 2, 128)])
@pytest.mark.parametrize("q_lens,kv_lens", [([64], [9000]), ([33, 100], [2500, 5000]), ([128, 17, 1], [4097, 700, 3000]),
                                            ([32, 130, 31], [6000, 6000, 1030])])
def test_tiles_cut_along_their_keys(hq, hkv, d, q_lens, kv_lens):
    # few items of up to a whole tile: more rows, fewer and longer pieces; the same bits every time
    b = batch(q_lens, kv_lens, hq, hkv, d, 32, seed=hq + d + 1)
    first = check(b, TOL_BF16)
    for _ in range(3):
        assert torch.equal(check(b, TOL_BF16).view(torch.int16), first.view(torch.int16))


def test_items_of_one_tile_between_items_of_two():
    # one CTA takes both kinds in turn; short items, so that one's end meets the next one's start
    q_lens = [64, 20, 33, 64, 7, 90] * 60
    kv_lens = [128, 100, 256, 30, 129, 64] * 60
    for _ in range(3):
        check(batch(q_lens, kv_lens, 16, 4, 128, 16, seed=14), TOL_BF16)


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (8, 2, 128), (32, 1, 128), (3, 3, 64)])
@pytest.mark.parametrize("q_lens,kv_lens", [([1], [513]), ([1, 2], [5000, 511]), ([8, 1, 0], [3000, 1, 9]), ([2, 9], [4097, 2048])])
def test_sequences_cut_along_their_keys(hq, hkv, d, q_lens, kv_lens):
    # few items: the keys of sequences of up to 32 rows are shared out, others stay whole
    check(batch(q_lens, kv_lens, hq, hkv, d, 32, seed=hq + d), TOL_BF16)


@pytest.mark.parametrize("d", [64, 128])
def test_output_at_any_16_byte_address(d):
    b = batch([300, 1, 40], [500, 700, 130], 8, 2, d, 16, seed=12)
    g, ref, n = b.to("cuda"), reference(b), b.num_tokens
    got = []
    for shift in (0, 8, 16):  # elements: 16 and 32 bytes
        room = torch.full((g.q.numel() + 24,), 7.0, dtype=BF16, device="cuda")
        out = room[shift:shift + g.q.numel()].view(g.q.shape)
        api.rpa_cross_forward(g.q, g.kv_pages, g.kv_lens, g.page_indices, g.cu_q_lens, g.num_seqs, sm_scale=b.sm_scale, out=out)
        assert (out[:n].cpu().double() - ref[:n]).abs().max().item() <= TOL_BF16
        assert (room[:shift] == 7.0).all() and (room[shift + n * 8 * d:] == 7.0).all()
        got.append(out[:n].clone())
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_no_sequences_and_one_stream_of_nothing():
    b = batch([2, 40], [30, 50], 8, 2, 128, 16, seed=1)
    b.num_seqs[0] = 0
    out, bits = run(b)
    assert bits == 0 and (out.float() == 7.0).all()


def test_extreme_logits_and_offsets():
    # logits of +-thousands, one key far above the rest at either end, equal keys
    b = batch([3, 50, 2], [900, 260, 900], 4, 2, 128, 16, seed=11)
    b.q[:] = (b.q.float() * 60).to(BF16)
    pages = b.kv_pages.view(-1, 4, 128)
    slot = lambda s, k: int(b.page_indices[s, k // 16]) * 16 + k % 16  # noqa: E731
    pages[slot(0, 899), 0::2] *= 8
    pages[slot(1, 0), 0::2] *= 8
    for k in range(900):
        pages[slot(2, k), 0::2] = pages[slot(2, 0), 0::2]
    check(b, TOL_BF16 * 2)  # one key's value dominates: outputs of up to 4 are rounded to 2^-8 of that


def test_kernel_timing_mode_and_batch_kinds_agree():
    b = batch(*LENS, 8, 2, 128, 16, seed=3)
    want = check(b, TOL_BF16)
    with api.KernelTimer() as kt:
        got, bits = run(b)
    # (timed kernels do not overlap, so the decode shares are cut elsewhere: equal up to rounding)
    n = b.num_tokens
    assert bits == 0 and (got[:n].double() - want[:n].double()).abs().max() <= TOL_BF16
    assert any(n.startswith("rpa_") for n in kt.result)
    e = batch([600, 1], [0, 0], 8, 2, 128, 16, seed=3)
    with api.KernelTimer():
        assert (run(e)[0][:601] == 0).all()
    dec = batch([1, 2, 4], [90, 0, 4000], 8, 2, 128, 16, seed=4)
    pre = batch([20, 70, 8], [90, 0, 4000], 8, 2, 128, 16, seed=4)
    for b, kind in ((dec, api.BATCH_DECODE_ONLY), (pre, api.BATCH_PREFILL_ONLY)):
        assert torch.equal(check(b, TOL_BF16, batch_kind=kind).view(torch.int16), check(b, TOL_BF16).view(torch.int16))
    out, bits = run(pre, batch_kind=api.BATCH_DECODE_ONLY)  # the excluded class is skipped and reported
    assert bits == 0x80 and (out[:20].float() == 7.0).all() and (out[90:98].float() == 7.0).all()


@pytest.mark.parametrize("what,code", [("kv_len", 0x04), ("negative kv_len", 0x04), ("huge kv_len", 0x04), ("page", 0x08),
                                       ("tokens", 0x10), ("num", 0x01)])
def test_bad_metadata_is_skipped_and_reported(what, code):
    b = batch([2, 40, 3], [100, 200, 50], 8, 2, 128, 16, seed=5)
    if what.endswith("kv_len"):
        b.kv_lens[1] = {"kv_len": 10**6, "negative kv_len": -3, "huge kv_len": 2**31 - 1}[what]
    elif what == "page":
        b.page_indices[1, 3] = 10**6
    elif what == "tokens":
        b.cu_q_lens[3] = 60
    else:
        b.num_seqs[0] = 9
    out, bits = run(b)
    assert bits == code
    ref = reference(batch([2, 40, 3], [100, 200, 50], 8, 2, 128, 16, seed=5))
    good = {"tokens": slice(0, 42), "num": slice(0, 0)}.get(what, [0, 1, 42, 43, 44])
    assert not out[good].numel() or (out[good].double() - ref[good]).abs().max() <= TOL_BF16
    if what != "page":  # (a bad page's keys are dropped from the rows that name it)
        rest = torch.ones(len(out), dtype=torch.bool)
        rest[good] = False
        assert (out[rest].float() == 7.0).all()


def test_refusals():
    b = batch([2, 5], [30, 4], 8, 2, 128, 16).to("cuda")
    good = dict(q=b.q, kv_pages=b.kv_pages, kv_lens=b.kv_lens, page_indices=b.page_indices, cu_q_lens=b.cu_q_lens,
                num_seqs=b.num_seqs)
    for bad in (dict(q=b.q.float()), dict(q=b.q[..., :64].contiguous()), dict(q=b.q.transpose(0, 1)), dict(kv_lens=b.kv_lens[:1]),
                dict(kv_lens=b.kv_lens.cpu()), dict(cu_q_lens=b.cu_q_lens[:2]), dict(out=b.q[:1].contiguous()), dict(q=b.q[:, 0])):
        with pytest.raises(ValueError):
            api.rpa_cross_forward(**{**good, **bad})
    for bad in (dict(sm_scale=math.nan), dict(soft_cap=math.inf), dict(out=b.q), dict(workspace=torch.zeros(512, dtype=torch.uint8, device="cuda")),
                dict(q=b.q[:, :7].contiguous())):
        with pytest.raises(api.RpaError):
            api.rpa_cross_forward(**{**good, **bad})
    assert api.rpa_cross_forward(**{**good, "q": b.q[:0]}).shape == (0, 8, 128)


def test_calls_on_two_streams_at_once():
    b1, b2 = batch([1] * 30 + [90], [2000] * 31, 8, 2, 128, 16, seed=1), batch([60] * 8, [900] * 8, 8, 2, 128, 16, seed=2)
    want = [check(b, TOL_BF16, workspace=False) for b in (b1, b2)]
    g = [b.to("cuda") for b in (b1, b2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [torch.full_like(b.q, 7.0) for b in g]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, b, out in zip(streams, g, outs):
            with torch.cuda.stream(st):
                api.rpa_cross_forward(b.q, b.kv_pages, b.kv_lens, b.page_indices, b.cu_q_lens, b.num_seqs,
                                      sm_scale=b.sm_scale, out=out)
    torch.cuda.synchronize()
    for out, ref in zip(outs, want):
        assert torch.equal(out.cpu().view(torch.int16), ref.view(torch.int16))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_calls_back_to_back_share_a_workspace(d):
    # calls on one stream, one workspace, nothing waits between them: different batches take turns
    bs = [batch([1] * 20 + [90], [1500] * 21, 8, 2, d, 16, seed=1), batch([60] * 8, [900] * 8, 8, 2, d, 16, seed=2),
          batch([2], [9000], 8, 2, d, 16, seed=3), batch([0, 5], [7, 0], 8, 2, d, 16, seed=4)]
    want = [check(b, TOL_BF16) for b in bs]
    g = [b.to("cuda") for b in bs]
    size = max(api.rpa_cross_workspace_size(api.make_rpa_params(b.q, b.kv_pages, b.page_indices)) for b in g)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    outs = [[torch.full_like(b.q, 7.0) for b in g] for _ in range(10)]
    torch.cuda.synchronize()
    for turn in outs:
        for b, out in zip(g, turn):
            api.rpa_cross_forward(b.q, b.kv_pages, b.kv_lens, b.page_indices, b.cu_q_lens, b.num_seqs, sm_scale=b.sm_scale,
                                  out=out, workspace=ws)
    assert api.check_device_status(ws) == 0
    for turn in outs:
        for out, ref in zip(turn, want):
            assert torch.equal(out.cpu().view(torch.int16), ref.view(torch.int16))


# ------------------------------------------------------------------ the fused step
def step_inputs(b, seed):
    """bf16 new rows for a batch whose cache may be narrower."""
    g = torch.Generator().manual_seed(seed)
    hkv = b.kv_pages.shape[2] // 2
    shape = (b.q.shape[0], hkv, b.q.shape[2])
    return torch.randn(shape, generator=g).to(BF16), torch.randn(shape, generator=g).to(BF16)


@pytest.mark.parametrize("dtype,ks,vs,kw", [
    (BF16, None, None, {}), (FP8, 0.03125, 0.0625, {}), (INT8, 0.03, 0.03, {}), (INT4, 0.4, 0.4, {}),
    (BF16, None, None, dict(sliding_window=50, soft_cap=20.0))], ids=str)
def test_step_is_the_write_then_attention(dtype, ks, vs, kw):
    b = batch([1, 1, 30, 5, 1, 200], [900, 1, 30, 77, 33, 450], 8, 2, 128, 16, dtype=dtype, seed=21, k_scale=ks, v_scale=vs, **kw)
    k, v = step_inputs(b, 4)
    t = api.make_rope_table(64, interleaved=True)
    g, k, v = b.to("cuda"), k.cuda(), v.cuda()
    meta = (g.kv_lens, g.page_indices, g.cu_q_lens, g.num_seqs)
    pages = g.kv_pages.clone()
    q_out, _ = api.rpa_rope_update_kv_cache(g.q, k, v, pages, *meta, t, k_scale=ks, v_scale=vs)
    want = api.rpa_forward(q_out, pages, *meta, out=torch.full_like(g.q, 7.0), **b.options())
    q_rot, out = torch.full_like(g.q, 5.0), torch.full_like(g.q, 7.0)
    ws = torch.zeros(api.rpa_workspace_size(api.make_rpa_params(g.q, g.kv_pages, g.page_indices, **b.options())),
                     dtype=torch.uint8, device="cuda")
    got = api.rpa_rope_forward_update(g.q, k, v, g.kv_pages, *meta, t, q_rot=q_rot, out=out, workspace=ws, **b.options())
    assert got is out and api.check_device_status(ws) == 0
    n = b.num_tokens
    assert torch.equal(g.kv_pages.view(torch.uint8), pages.view(torch.uint8))
    assert torch.equal(q_rot[:n].view(torch.int16), q_out[:n].view(torch.int16)) and (q_rot[n:].float() == 5.0).all()
    # (the step may cut decode's keys elsewhere than rpa_forward does: equal up to rounding)
    tol = (TOL_BF16 if dtype == BF16 else TOL_FP8) * (3 if dtype in (INT8, INT4) else 1)
    assert (out[:n].double() - want[:n].double()).abs().max().item() <= tol and (out[n:].float() == 7.0).all()
    # and against the oracle, which attends over the cache as written
    ref = oracle.rpa(q_rot.cpu(), g.kv_pages.cpu(), b.kv_lens, b.page_indices, b.cu_q_lens, len(b.q_lens), **b.options())
    err = (out[:n].cpu().double() - ref[:n]).abs().max().item()
    assert err <= tol


@pytest.mark.parametrize("dtype,ks,vs", [(BF16, None, None), (FP8, None, None), (FP8, 0.5, 0.25)], ids=str)
@pytest.mark.parametrize("hq,hkv,d,ps", [(12, 2, 64, 16), (64, 8, 256, 8), (8, 4, 128, 16), (16, 16, 128, 64)])
def test_step_of_small_decode_batches(dtype, ks, vs, hq, hkv, d, ps):
    """Decode shares shorter than rpa_forward's: batches whose shares are as short as they get, on one
    workspace that each leaves its lists in for the next."""
    t = api.make_rope_table(d)
    lens = [([1] * 24, list(range(20, 2000, 83))), ([1] * 4 + [23], [2788, 300, 16, 1100, 523]), ([1], [129]), ([1] * 9, [1] * 9),
            ([2, 1, 1], [640, 128, 127]), ([1] * 40, [150] * 40), ([1], [5000])]
    ws = torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")
    for i, (q_lens, kv_lens) in enumerate(lens):
        b = batch(q_lens, kv_lens, hq, hkv, d, ps, dtype=dtype, seed=40 + i, k_scale=ks, v_scale=vs)
        k, v = step_inputs(b, i)
        g, k, v = b.to("cuda"), k.cuda(), v.cuda()
        meta = (g.kv_lens, g.page_indices, g.cu_q_lens, g.num_seqs)
        q_rot, out = torch.empty_like(g.q), torch.full_like(g.q, 7.0)
        for _ in range(2):  # (the same rows again: the same cache)
            out.fill_(7.0)
            api.rpa_rope_forward_update(g.q, k, v, g.kv_pages, *meta, t, q_rot=q_rot, out=out, workspace=ws, **b.options())
        assert api.check_device_status(ws) == 0
        n = b.num_tokens
        ref = oracle.rpa(q_rot.cpu(), g.kv_pages.cpu(), b.kv_lens, b.page_indices, b.cu_q_lens, len(b.q_lens), **b.options())
        err = (out[:n].cpu().double() - ref[:n]).abs().max().item()
        assert err <= (TOL_BF16 if dtype == BF16 else TOL_FP8), (i, err)
        assert (out[n:].float() == 7.0).all()


def test_step_reports_bad_metadata_and_refuses():
    b = batch([1, 4], [30, 20], 8, 2, 128, 16, seed=2)
    k, v = (x.cuda() for x in step_inputs(b, 1))
    t, g = api.make_rope_table(128), b.to("cuda")
    meta = (g.kv_lens, g.page_indices, g.cu_q_lens, g.num_seqs)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    g.kv_lens[1] = 3
    api.rpa_rope_forward_update(g.q, k, v, g.kv_pages, *meta, t, workspace=ws, sm_scale=0.1)
    assert api.check_device_status(ws) == 0x02
    with pytest.raises(ValueError):
        api.rpa_rope_forward_update(None, k, v, g.kv_pages, *meta, t)
    with pytest.raises(ValueError):
        api.rpa_rope_forward_update(g.q, k, v, g.kv_pages, *meta, t, out=g.q[:2].contiguous())
    for kw in (dict(out=g.q), dict(workspace=ws[:512]), dict(sliding_window=-1)):
        with pytest.raises(api.RpaError):
            api.rpa_rope_forward_update(g.q, k, v, g.kv_pages, *meta, t, **kw)


def test_all_attention_calls_share_a_workspace():
    # causal, cross and step take turns on one workspace, nothing waits between them
    b = batch([1] * 20 + [90, 7], [1500] * 21 + [600], 8, 2, 128, 16, seed=31)
    e = batch([3, 200, 1], [70, 900, 5000], 8, 2, 128, 16, seed=32)
    k, v = step_inputs(b, 5)
    g, ge, k, v = b.to("cuda"), e.to("cuda"), k.cuda(), v.cuda()
    t, size = api.make_rope_table(128), 1 << 27
    meta = lambda x: (x.kv_lens, x.page_indices, x.cu_q_lens, x.num_seqs)  # noqa: E731
    calls = [lambda out, ws: api.rpa_forward(g.q, g.kv_pages, *meta(g), sm_scale=b.sm_scale, out=out, workspace=ws),
             lambda out, ws: api.rpa_cross_forward(ge.q, ge.kv_pages, *meta(ge), sm_scale=e.sm_scale, out=out, workspace=ws),
             lambda out, ws: api.rpa_rope_forward_update(g.q, k, v, g.kv_pages, *meta(g), t, sm_scale=b.sm_scale, out=out, workspace=ws),
             lambda out, ws: api.rpa_cross_forward(g.q, g.kv_pages, *meta(g), sm_scale=b.sm_scale, out=out, workspace=ws)]
    qs = [g.q, ge.q, g.q, g.q]
    fresh = lambda: torch.zeros(size, dtype=torch.uint8, device="cuda")  # noqa: E731
    calls[2](torch.empty_like(g.q), fresh())  # (the step's rows are written: the cache stays as it is from here on)
    torch.cuda.synchronize()
    want = []
    for call, q in zip(calls, qs):
        want.append(call(torch.full_like(q, 7.0), fresh()))
        torch.cuda.synchronize()
    ws, outs = fresh(), [[torch.full_like(q, 7.0) for q in qs] for _ in range(8)]
    torch.cuda.synchronize()
    for i, turn in enumerate(outs):
        for j in range(4):
            c = (i + j * (1 + 2 * (i % 2))) % 4
            calls[c](turn[c], ws)
    assert api.check_device_status(ws) == 0
    for turn in outs:
        for out, ref in zip(turn, want):
            assert torch.equal(out.view(torch.int16), ref.view(torch.int16))


@pytest.mark.parametrize("d,dtype,scale", [(64, BF16, None), (128, BF16, None), (128, FP8, 0.5)], ids=str)
def test_replays_follow_what_the_tensors_hold(d, dtype, scale):
    """Captured once, replayed on other batches written into the same tensors; two graphs in turn."""
    hq, hkv, ps, tokens, seqs, pages = 8, 2, 16, 160, 8, 400
    rng = np.random.default_rng(7)
    cuda = lambda *shape, **kw: torch.zeros(*shape, device="cuda", **kw)  # noqa: E731
    i32 = torch.int32
    q, k, v = (cuda(tokens, h, d, dtype=BF16) for h in (hq, hkv, hkv))
    kv = torch.from_numpy(rng.standard_normal((pages, ps, 2 * hkv, d), dtype=np.float32)).to(dtype).cuda()
    lens, cu, num = cuda(seqs, dtype=i32), cuda(seqs + 1, dtype=i32), cuda(1, dtype=i32)
    tbl = torch.from_numpy(rng.permutation(pages)[:seqs * (pages // seqs)].reshape(seqs, -1).astype(np.int32)).cuda().contiguous()
    meta, t = (lens, tbl, cu, num), api.make_rope_table(d)
    outs = [torch.full_like(q, 7.0) for _ in range(2)]
    run = [lambda out: api.rpa_cross_forward(q, kv, *meta, sm_scale=0.1, k_scale=scale, v_scale=scale, out=out),
           lambda out: api.rpa_rope_forward_update(q, k, v, kv, *meta, t, sm_scale=0.1, k_scale=scale, v_scale=scale, out=out)]
    graphs = []
    for f, out in zip(run, outs):
        f(out)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f(out)
    batches = [([1] * 8, [700, 3, 90, 512, 1, 33, 600, 799]), ([150, 1], [400, 20]), ([], []), ([2, 0, 40, 60], [300, 50, 41, 60])]
    for q_lens, kv_lens in batches * 2:
        n = len(q_lens)
        for x in (q, k, v):
            x.copy_(torch.from_numpy(rng.standard_normal(tuple(x.shape), dtype=np.float32)).to(BF16))
        lens[:n] = torch.tensor(kv_lens, dtype=i32)
        cu[:n + 1] = torch.tensor([0] + list(np.cumsum(q_lens)), dtype=i32)
        num[0] = n
        for out in outs:
            out.fill_(7.0)
        for g in graphs[::-1]:  # (the step writes its rows first)
            g.replay()
        for out, f in zip(outs, run):
            want = torch.full_like(q, 7.0)
            f(want)
            assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        m = sum(q_lens)
        ref = plain.attend_all(q.cpu(), kv.cpu(), lens.cpu(), tbl.cpu(), cu.cpu(), n, sm_scale=0.1, k_scale=scale, v_scale=scale)
        tol = TOL_BF16 if dtype == BF16 else TOL_FP8
        assert m == 0 or (outs[0][:m].cpu().double() - ref[:m]).abs().max().item() <= tol
        assert (outs[0][m:].float() == 7.0).all() and (outs[1][m:].float() == 7.0).all()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_decoder_layer(graph):
    d, hq, hkv, ps = 64, 4, 2, 16
    enc_lens, dec_lens, new = [70, 0, 33], [9, 20, 1], [1, 20, 1]
    rng = np.random.default_rng(3)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    rand = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32)).to(BF16)  # noqa: E731
    # the encoder's states go into pages of their own, unturned, in e4m3 halves of their size
    enc = batch(enc_lens, enc_lens, hkv, hkv, d, ps, dtype=FP8, seed=8, pad=0)
    ek, ev = rand(sum(enc_lens), hkv, d), rand(sum(enc_lens), hkv, d)
    ge = enc.to("cuda")
    api.rpa_rope_update_kv_cache(None, ek.cuda(), ev.cuda(), ge.kv_pages, ge.kv_lens, ge.page_indices, ge.cu_q_lens, ge.num_seqs,
                                 api.make_rope_table(0), k_scale=0.0625, v_scale=0.0625)
    dec = batch(new, dec_lens, hq, hkv, d, ps, seed=9, pad=1)
    gd = dec.to("cuda")
    k, v = step_inputs(dec, 6)
    x = dict(q=gd.q, k=k.cuda(), v=v.cuda(), q_rot=torch.zeros_like(gd.q), y=torch.zeros_like(gd.q), z=torch.zeros_like(gd.q))
    table = api.make_rope_table(32, scaling={"type": "linear", "factor": 2.0})
    ws = [torch.zeros(1 << 26, dtype=torch.uint8, device="cuda") for _ in range(2)] if not graph else [None, None]

    def cross(y):
        enc_meta = (ge.kv_lens, ge.page_indices, gd.cu_q_lens, gd.num_seqs)
        return api.rpa_cross_forward(y, ge.kv_pages, *enc_meta, sm_scale=0.125, k_scale=0.0625, v_scale=0.0625, out=x["z"], workspace=ws[1])

    def layer():
        y = api.rpa_rope_forward_update(x["q"], x["k"], x["v"], gd.kv_pages, gd.kv_lens, gd.page_indices, gd.cu_q_lens, gd.num_seqs,
                                        table, sm_scale=0.125, q_rot=x["q_rot"], out=x["y"], workspace=ws[0])
        return cross(y)

    layer()
    torch.cuda.synchronize()
    if graph:
        eager = x["z"].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer()
        x["z"].zero_()
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(x["z"].view(torch.int16), eager.view(torch.int16))
    else:
        assert api.check_device_status(ws[0]) == 0 and api.check_device_status(ws[1]) == 0
    # float64, from the definitions: the rotated rows rounded once, causal attention, all encoder keys
    f, amp = plain.frequencies(32, 10000.0, {"type": "linear", "factor": 2.0})
    n = sum(new)
    pos = torch.cat([torch.arange(L - m, L) for L, m in zip(dec_lens, new)])
    q = plain.rope(dec.q[:n], pos, f, amp, False).to(BF16)
    flat = dec.kv_pages.clone()
    seq = torch.cat([torch.full((m,), s) for s, m in enumerate(new)])
    slot = dec.page_indices[seq, pos // ps].long() * ps + pos % ps
    flat.view(-1, 2 * hkv, d)[slot, 0::2] = plain.rope(k[:n], pos, f, amp, False).to(BF16)
    flat.view(-1, 2 * hkv, d)[slot, 1::2] = v[:n]
    full = torch.cat([q, dec.q[n:]])
    y = oracle.rpa(full, flat, dec.kv_lens, dec.page_indices, dec.cu_q_lens, len(new), sm_scale=0.125)
    assert (x["y"][:n].cpu().double() - y[:n]).abs().max() <= TOL_BF16
    z = plain.attend_all(x["y"].cpu(), ge.kv_pages.cpu(), enc.kv_lens, enc.page_indices, dec.cu_q_lens, len(new), sm_scale=0.125,
                         k_scale=0.0625, v_scale=0.0625)
    assert (x["z"][:n].cpu().double() - z[:n]).abs().max() <= TOL_FP8
    # the e4m3 states are within half a step of the states themselves
    at = torch.cat([ge.page_indices.cpu()[s, torch.arange(L) // ps].long() * ps + torch.arange(L) % ps for s, L in enumerate(enc_lens)])
    held = ge.kv_pages.cpu().view(torch.uint8).flatten(0, 1)[at].view(FP8).double() * 0.0625
    for part, src in ((0, ek), (1, ev)):
        assert ((held[:, part::2] - src.double()).abs() <= src.double().abs() * 2.0 ** -4 + 2.0 ** -10 * 0.0625 + 1e-6).all()


def test_latent_attention_with_turned_rope_parts():
    # rope_apply in front of mla_rpa_forward: q_pe and new_k_pe turned in place, then the call's own write
    m = workloads.make_mla([1, 3], [40, 9], seed=5, page_size=16, max_num_tokens=6)
    dist = m.to("cuda")
    t = api.make_rope_table(64, interleaved=True, scaling={"type": "yarn", "factor": 40.0, "original_max_position": 4096})
    f, amp = plain.frequencies(64, 10000.0, {"type": "yarn", "factor": 40.0, "original_max_position": 4096})
    pos = torch.tensor([39, 6, 7, 8, 0, 0], dtype=torch.int32)
    api.rope_apply(dist.q_pe, dist.new_k_pe[:, None], pos.cuda(), t, q_out=dist.q_pe, k_out=dist.new_k_pe[:, None])
    out = api.mla_rpa_forward(dist.ql_nope, dist.q_pe, dist.new_kv_c, dist.new_k_pe, dist.cache_kv_c, dist.cache_k_pe, dist.kv_lens,
                              dist.page_indices, dist.cu_q_lens, dist.distribution, **m.options())
    m.q_pe[:4] = plain.rope(m.q_pe[:4], pos[:4], f, amp, True).to(BF16)
    m.new_k_pe[:4] = plain.rope(m.new_k_pe[:4, None], pos[:4], f, amp, True)[:, 0].to(BF16)
    ref, _, _ = oracle.mla_forward(m.ql_nope, m.q_pe, m.new_kv_c, m.new_k_pe, m.cache_kv_c, m.cache_k_pe, m.kv_lens,
                                   m.page_indices, m.cu_q_lens, m.distribution, **m.options())
    assert (out[:4].cpu().double() - ref[:4]).abs().max() <= TOL_BF16
