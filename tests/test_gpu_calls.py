"""Calls of the rotating, appending and cross-attention operators that their documentation allows and that
the parity tests beside this file do not make."""
import threading

import pytest
import torch

import plain
from parity import TOL_BF16
from ragged_paged_attention_gb300 import api
from test_gpu_cross import batch, reference
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
