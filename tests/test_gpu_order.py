"""Calls behind a kernel of the caller's that writes their metadata, and lets them start before it has
(tests/late_writer.cu): they see what it wrote, in a stream and in a graph."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from ragged_paged_attention_gb300 import api
from ragged_paged_attention_gb300 import build as rpa_build

pytestmark = pytest.mark.gpu

BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn
SEQS, TOKENS = 6, 96
# (q_lens, kv_lens): lengths, counts and empty sequences change between the two; both are good everywhere
OLD = [1, 1, 40, 0, 2, 1], [30, 200, 70, 9, 500, 1]
NEW = [3, 20, 1, 60], [300, 20, 513, 70]
OLD_CROSS = [1, 0, 40, 3, 2, 1], [0, 200, 0, 9, 500, 1]
NEW_CROSS = [3, 20, 1, 60], [300, 0, 513, 5]


@pytest.fixture(scope="module")
def late_write(tmp_path_factory):
    so = tmp_path_factory.mktemp("late") / "late_writer.so"
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "late_writer.cu")
    subprocess.run([rpa_build._nvcc(), *rpa_build.ARCH, "-O2", "-shared", "-Xcompiler", "-fPIC", "-o", str(so), src], check=True)
    f = ctypes.CDLL(str(so)).late_write
    f.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]

    def write(dst, src):
        assert dst.numel() == src.numel()
        assert f(dst.data_ptr(), src.data_ptr(), dst.numel(), 60, torch.cuda.current_stream().cuda_stream) == 0
    return write


def metadata(q_lens, kv_lens):
    """kv_lens, cu_q_lens and num_seqs in one int32 tensor."""
    m = np.zeros(2 * SEQS + 2, np.int32)
    m[:len(kv_lens)] = kv_lens
    m[SEQS:SEQS + len(q_lens) + 1] = np.concatenate([[0], np.cumsum(q_lens)])
    m[-1] = len(q_lens)
    return torch.from_numpy(m).cuda()


def parts(m):
    return m[:SEQS], m[SEQS:2 * SEQS + 1], m[2 * SEQS + 1:]


@pytest.mark.parametrize("graph", [False, True], ids=["stream", "graph"])
@pytest.mark.parametrize("call", ["cross", "forward", "update", "step"])
@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, BF16), (256, BF16), (128, FP8)], ids=str)
def test_lengths_written_just_before_the_call(late_write, call, d, dtype, graph):
    hq, hkv, ps = 8, 2, 16
    rng = np.random.default_rng(d)
    rand = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32))  # noqa: E731
    pages = SEQS * 40
    kv = rand(pages, ps, 2 * hkv, d).to(dtype).cuda()
    q, k, v = (rand(TOKENS, h, d).to(BF16).cuda() for h in (hq, hkv, hkv))
    tbl = torch.from_numpy(rng.permutation(pages).astype(np.int32)).cuda().view(SEQS, -1)
    table = api.make_rope_table(64)
    old, new = (metadata(*x) for x in ((OLD_CROSS, NEW_CROSS) if call == "cross" else (OLD, NEW)))
    held = old.clone()
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")

    def run(m, cache, out):
        lens, cu, num = parts(m)
        kw = dict(sm_scale=0.1, out=out, workspace=ws)
        if call == "cross":
            api.rpa_cross_forward(q, cache, lens, tbl, cu, num, **kw)
        elif call == "forward":
            api.rpa_forward(q, cache, lens, tbl, cu, num, **kw)
        elif call == "update":
            api.rpa_forward_update(q, k.to(dtype), v.to(dtype), cache, lens, tbl, cu, num, **kw)
        else:
            api.rpa_rope_forward_update(q, k, v, cache, lens, tbl, cu, num, table, k_scale=None, **kw)

    want, want_kv = torch.full_like(q, 7.0), kv.clone()
    run(new, want_kv, want)
    torch.cuda.synchronize()
    out, got_kv = torch.full_like(q, 7.0), kv.clone()

    def both():
        late_write(held, new)
        run(held, got_kv, out)

    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            both()
        both = g.replay
    for _ in range(5):
        held.copy_(old)
        got_kv.view(torch.uint8).copy_(kv.view(torch.uint8))
        out.fill_(7.0)
        torch.cuda.synchronize()
        both()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        assert torch.equal(got_kv.view(torch.uint8), want_kv.view(torch.uint8))
    assert api.check_device_status(ws) == 0
