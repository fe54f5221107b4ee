"""Calls of the rotating, appending and cross-attention operators that their documentation allows and that
the parity tests beside this file do not make."""
import ctypes
import math
import threading

import pytest
import torch

import oracle
import plain
from parity import TOL_BF16, TOL_FP8
from ragged_paged_attention_gb300 import api
from test_gpu_cross import batch, check, reference, step_inputs
from test_gpu_rope import bits, near, randn

pytestmark = pytest.mark.gpu

BF16, FP8, INT8, INT4 = torch.bfloat16, torch.float8_e4m3fn, torch.int8, torch.uint8


@pytest.mark.parametrize("T,H", [(1, 1), (1, 5), (19, 1), (19, 5), (300, 16)])
@pytest.mark.parametrize("rot,inter", [(64, False), (48, True), (24, False), (6, True)])
def test_parts_of_the_same_heads_in_place(T, H, rot, inter):
    # [T, H, 3, D]: q and k of a head beside one another, turned where they are; v stays
    x = randn(T + H, T, H, 3, 64)
    g, pos = x.cuda(), torch.arange(5, 5 + T, dtype=torch.int32)
    t, (f, amp) = api.make_rope_table(rot, interleaved=inter), plain.frequencies(rot)
    q, k = g[:, :, 0], g[:, :, 1]
    api.rope_apply(q, k, pos.cuda(), t, q_out=q, k_out=k)
    for i in (0, 1):
        near(g[:, :, i].cpu(), plain.rope(x[:, :, i], pos, f, amp, inter), plain.rope_slack(x[:, :, i], f, amp, inter))
    assert torch.equal(bits(g[:, :, 2].cpu()), bits(x[:, :, 2]))
    # q's result into v's place, k's into q's
    g = x.cuda()
    with pytest.raises(api.RpaError):
        api.rope_apply(g[:, :, 0], g[:, :, 1], pos.cuda(), t, q_out=g[:, :, 2], k_out=g[:, :, 0])
    api.rope_apply(g[:, :, 0], None, pos.cuda(), t, q_out=g[:, :, 2])
    near(g[:, :, 2].cpu(), plain.rope(x[:, :, 0], pos, f, amp, inter), plain.rope_slack(x[:, :, 0], f, amp, inter))
    assert torch.equal(bits(g[:, :, :2].cpu()), bits(x[:, :, :2]))


# ------------------------------------------------------------------ workspaces of calls that were given none
def cross(b, g, **kw):
    return api.rpa_cross_forward(g.q, g.kv_pages, g.kv_lens, g.page_indices, g.cu_q_lens, g.num_seqs, sm_scale=b.sm_scale, **kw)


def test_own_workspaces_go_with_their_thread():
    b = batch([1, 20], [300, 64], 8, 2, 128, 16, seed=1)
    g, ref, n = b.to("cuda"), reference(b), b.num_tokens
    outs, all_called = [], threading.Barrier(4)

    def work(stream):
        with torch.cuda.stream(stream):
            outs.append(cross(b, g))
        stream.synchronize()
        all_called.wait(60)

    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    threads = [threading.Thread(target=work, args=(torch.cuda.Stream(),)) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    size = api.rpa_cross_workspace_size(api.make_rpa_params(g.q, g.kv_pages, g.page_indices))
    assert torch.cuda.memory_allocated() - before < size  # (four outputs of some KB)
    for out in outs:
        assert (out[:n].cpu().double() - ref[:n]).abs().max().item() <= TOL_BF16


def test_the_error_word_of_an_own_workspace():
    b = batch([2, 40, 3], [100, 200, 50], 8, 2, 128, 16, seed=5)
    b.kv_lens[1] = 10**6
    g = b.to("cuda")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    with torch.cuda.stream(streams[0]):
        cross(b, g)
        seen = []
        t = threading.Thread(target=lambda: seen.append(api.check_device_status()))  # that thread has made no call
        t.start()
        t.join()
    with torch.cuda.stream(streams[1]):
        seen.append(api.check_device_status())  # nor has this stream seen one of ours
    with torch.cuda.stream(streams[0]):
        seen += [api.check_device_status(), api.check_device_status()]
    assert seen == [0, 0, 0x04, 0]


def test_a_graph_of_a_call_with_the_shared_workspace_after_a_larger_call():
    b, big = batch([1, 20], [300, 64], 8, 2, 128, 16, seed=1), batch([1] * 900, [40] * 900, 32, 16, 256, 16, seed=2)
    g, n = b.to("cuda"), b.num_tokens
    run = lambda b, g, out: api.rpa_forward(g.q, g.kv_pages, g.kv_lens, g.page_indices, g.cu_q_lens, g.num_seqs, out=out, **b.options())  # noqa: E731
    want, out = run(b, g, torch.full_like(g.q, 7.0)), torch.full_like(g.q, 7.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(b, g, out)
    gb = big.to("cuda")
    run(big, gb, torch.empty_like(gb.q))
    torch.cuda.synchronize()
    filler = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(200)]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(out[:n]), bits(want[:n])) and all((f == 255).all() for f in filler)


# ------------------------------------------------------------------ cross attention
LENS = ([1, 3, 0, 2, 40, 1, 150, 17, 5], [1, 700, 64, 0, 9, 1500, 130, 0, 600])


@pytest.mark.parametrize("scale", [-0.125, -1.5, 0.0, 1e-30])
@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, BF16), (256, BF16), (128, FP8), (128, INT4)], ids=str)
def test_scales_of_either_sign(scale, d, dtype):
    b = batch(*LENS, 8, 2, d, 16, dtype=dtype, seed=d, sm_scale=scale)
    check(b, (TOL_BF16 if dtype == BF16 else TOL_FP8) * (4 if dtype == INT4 else 1))  # (int4 values are up to 8)


@pytest.mark.parametrize("hq,hkv", [(6, 1), (12, 2), (40, 5), (48, 1), (71, 1), (128, 1), (160, 1), (16, 16)])
@pytest.mark.parametrize("d,dtype,ks", [(64, BF16, None), (128, BF16, None), (128, FP8, None), (64, FP8, 0.37), (256, INT8, 2.0**-6)],
                         ids=str)
def test_group_sizes(hq, hkv, d, dtype, ks):
    b = batch(*LENS, hq, hkv, d, 16, dtype=dtype, seed=hq, k_scale=ks, v_scale=ks)
    check(b, TOL_BF16 if dtype == BF16 else TOL_FP8)  # (int8 values times 2^-6 are up to 2)


@pytest.mark.parametrize("ps", [1, 24, 256, 1024])
@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, BF16), (128, FP8)], ids=str)
def test_page_sizes(ps, d, dtype):
    check(batch(*LENS, 8, 2, d, ps, dtype=dtype, seed=ps), TOL_BF16 if dtype == BF16 else TOL_FP8)


def test_a_soft_cap_below_zero_and_one_beside_a_negative_scale():
    check(batch(*LENS, 4, 2, 128, 16, seed=3, soft_cap=-20.0), TOL_BF16)  # cap tanh(x / cap) is even in cap
    check(batch(*LENS, 4, 2, 64, 16, seed=3, soft_cap=3.0, sm_scale=-0.3), TOL_BF16)


@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, BF16), (128, FP8)], ids=str)
def test_sequences_that_share_pages(d, dtype):
    # one encoder's states read by many sequences, each to a length of its own; a page twice in one sequence
    kv_lens = [1200, 1, 700, 1200, 16, 1199, 900, 333]
    b = batch([1, 30, 2, 64, 1, 1, 200, 4], kv_lens, 8, 2, d, 16, dtype=dtype, seed=6)
    b.page_indices[1:len(kv_lens)] = b.page_indices[0]
    b.page_indices[6, 3] = b.page_indices[6, 20]
    check(b, TOL_BF16 if dtype == BF16 else TOL_FP8)


@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, BF16), (64, FP8)], ids=str)
def test_one_long_sequence_among_many_short_ones(d, dtype):
    n = 160
    q_lens, kv_lens = [1] * n, [10 + s % 30 for s in range(n)]
    kv_lens[77], q_lens[78] = 9000, 70
    check(batch(q_lens, kv_lens, 8, 4, d, 16, dtype=dtype, seed=2), TOL_BF16 if dtype == BF16 else TOL_FP8)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_most_slots_of_the_tables_unused(d):
    b = batch([2, 40], [300, 1000], 8, 2, d, 16, seed=4)
    wide = batch([2, 40] + [0] * 3000, [300, 1000] + [0] * 3000, 8, 2, d, 16, seed=4)
    wide.num_seqs[0] = 2
    g, w = b.to("cuda"), wide.to("cuda")
    n = b.num_tokens
    assert torch.equal(bits(cross(b, g)[:n]), bits(cross(wide, w)[:n]))


# ------------------------------------------------------------------ a caller's own table
@pytest.mark.parametrize("rot,inter", [(64, False), (32, True), (20, False), (6, True)])
def test_frequencies_of_the_callers_own(rot, inter):
    # any turn per position, more than a whole one and backwards among them; amplitude negative and 0
    gen = torch.Generator().manual_seed(rot)
    turns = (torch.rand(rot // 2, generator=gen, dtype=torch.float64) * 4 - 2)
    steps = [int(round(float(x) * 2**64)) % 2**64 for x in turns]
    f = torch.tensor([(s if s < 2**63 else s - 2**64) / 2.0**64 for s in steps], dtype=torch.float64) * 2 * math.pi
    # (positions below 2^20: the float64 angle of the form itself is within 2^20 * 2^-50 of the table's)
    pos = torch.tensor([0, 1, -1, 77, 4095, -1000, 2**20 - 1, 3], dtype=torch.int32)
    x = randn(rot, len(pos), 3, 64)
    for amp in (1.0, -0.5, 0.0, 3.0):
        t = api.rope_table(struct_size=ctypes.sizeof(api.rope_table), version=1, rotary_dim=rot, pairing=int(inter), amplitude=amp)
        for i, s in enumerate(steps):
            t.step[i] = s
        for inverse in (False, True):
            out, _ = api.rope_apply(x.cuda(), None, pos.cuda(), t, inverse=inverse)
            near(out.cpu(), plain.rope(x, pos, f, amp, inter, inverse), plain.rope_slack(x, f, amp, inter))


# ------------------------------------------------------------------ the step
@pytest.mark.parametrize("dtype,scale", [(BF16, None), (FP8, 0.0625), (INT8, 0.03), (INT4, 0.4)], ids=str)
@pytest.mark.parametrize("hq,hkv,d,ps", [(8, 2, 128, 16), (12, 2, 64, 24), (9, 3, 256, 8)])
def test_short_chunks_over_long_contexts(dtype, scale, hq, hkv, d, ps):
    q_lens, kv_lens = [20, 1, 70, 3, 1], [4000, 3999, 2500, 1700, 5]
    b = batch(q_lens, kv_lens, hq, hkv, d, ps, dtype=dtype, seed=hq, k_scale=scale, v_scale=scale)
    k, v = step_inputs(b, 3)
    t = api.make_rope_table(d // 2)
    g, k, v = b.to("cuda"), k.cuda(), v.cuda()
    q_rot, out = torch.full_like(g.q, 5.0), torch.full_like(g.q, 7.0)
    api.rpa_rope_forward_update(g.q, k, v, g.kv_pages, g.kv_lens, g.page_indices, g.cu_q_lens, g.num_seqs, t, q_rot=q_rot, out=out,
                                **b.options())
    assert api.check_device_status() == 0
    n = b.num_tokens
    ref = oracle.rpa(q_rot.cpu(), g.kv_pages.cpu(), b.kv_lens, b.page_indices, b.cu_q_lens, len(q_lens), **b.options())
    # (int8 and int4 values are up to 127 and 8: outputs of up to about 4 after the scale)
    tol = TOL_BF16 if dtype == BF16 else TOL_FP8 * (3 if dtype in (INT8, INT4) else 1)
    assert (out[:n].cpu().double() - ref[:n]).abs().max().item() <= tol
    assert (out[n:].float() == 7.0).all() and (q_rot[n:].float() == 5.0).all()


def test_the_step_of_one_class_and_of_queries_in_place():
    t = api.make_rope_table(128)
    for q_lens, kv_lens, kind in (([1, 2, 4], [90, 3, 4000], api.BATCH_DECODE_ONLY), ([20, 70, 8], [90, 70, 4000], api.BATCH_PREFILL_ONLY)):
        b = batch(q_lens, kv_lens, 8, 2, 128, 16, seed=4)
        k, v = step_inputs(b, 2)
        got = []
        for kw in (dict(batch_kind=kind), dict()):
            g = b.to("cuda")
            g.kv_pages = g.kv_pages.clone()
            q = g.q.clone()
            out = torch.full_like(q, 7.0)
            api.rpa_rope_forward_update(q, k.cuda(), v.cuda(), g.kv_pages, g.kv_lens, g.page_indices, g.cu_q_lens, g.num_seqs, t,
                                        q_rot=q, out=out, sm_scale=b.sm_scale, **kw)
            assert api.check_device_status() == 0
            got.append((q, out, g.kv_pages))
        n = b.num_tokens
        assert torch.equal(bits(got[0][0]), bits(got[1][0])) and torch.equal(bits(got[0][2]), bits(got[1][2]))
        ref = oracle.rpa(got[0][0].cpu(), got[0][2].cpu(), b.kv_lens, b.page_indices, b.cu_q_lens, len(q_lens), sm_scale=b.sm_scale)
        for _, out, _ in got:
            assert (out[:n].cpu().double() - ref[:n]).abs().max().item() <= TOL_BF16
            assert (out[n:].float() == 7.0).all()
