"""The operators of a long context behind late writers, on streams of their own and in graphs that share a workspace: what
each gives is what it gives alone, bit by bit."""
import pytest
import torch

from long_context import BF16, Batch
from ragged_paged_attention_gb300 import api

pytestmark = pytest.mark.gpu

BATCHES = {"decodes": ([1, 2, 1, 1], [700, 300, 1, 900]), "prompts": ([40, 1, 300, 65], [640, 200, 300, 65])}


class Step:
    """One of each call over a batch, in the order of use, on inputs that may be written late."""

    def __init__(self, b, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.b, n = b, len(b.kv_lens)
        t = b.q.shape[0]
        rand = lambda *s: torch.randn(*s, generator=g).to(BF16)  # noqa: E731
        kv, lens, pages, cu, num = (x.cpu() for x in b.gpu())
        self.host = dict(kv=kv, lens=lens, pages=pages, cu=cu, num=num, q=rand(t, b.hq, b.d), k=rand(t, b.hkv, b.d), v=rand(t, b.hkv, b.d),
                         w=torch.rand(b.total, b.hkv, b.ps, generator=g), budgets=torch.full((n,), 96, dtype=torch.int32))
        self.source = {k: v.cuda() for k, v in self.host.items()}
        # what a kernel reads before its inputs are written: no sequences, lengths and pages that are refused
        self.dev = {k: torch.zeros_like(v) for k, v in self.source.items()}
        prm = api.make_g4_params(self.dev["q"], self.dev["kv"], self.dev["pages"])
        kw = api._batch_params(self.dev["q"].get_device(), t, b.hq, b.d, self.dev["kv"], *(self.dev[k] for k in ("lens", "pages", "cu", "num")), g4=True)
        ev = api.make_evict_params(self.dev["kv"], self.dev["pages"], 96, sinks=2, recent=8)
        self.bytes = max(api.rpa_g4_workspace_size(prm), api.rpa_key_weights_workspace_size(kw), api.rpa_evict_workspace_size(ev))
        self.table = api.make_rope_table(b.d)

    def workspace(self):
        return torch.zeros(self.bytes, dtype=torch.uint8, device="cuda")

    def write(self):
        for k, v in self.source.items():
            self.dev[k].copy_(v, non_blocking=True)

    def run(self, ws):
        x, b = self.dev, self.b
        t = x["q"].shape[0]
        q = torch.zeros_like(x["q"])
        api.rpa_g4_update_kv_cache(x["q"], x["k"], x["v"], x["kv"], x["lens"], x["pages"], x["cu"], x["num"], self.table, q_out=q, workspace=ws)
        k, v = (torch.zeros(t, b.hkv, b.d, dtype=BF16, device="cuda") for _ in range(2))
        api.rpa_g4_read_kv_cache(x["kv"], x["lens"], x["pages"], x["cu"], x["num"], k_out=k, v_out=v, workspace=ws)
        out = api.rpa_g4_forward(q, x["kv"], x["lens"], x["pages"], x["cu"], x["num"], sm_scale=b.d ** -0.5, out=torch.zeros_like(q), workspace=ws)
        w = api.rpa_key_weights(q, x["kv"], x["lens"], x["pages"], x["cu"], x["num"], x["w"], sm_scale=b.d ** -0.5, workspace=ws)
        slots = torch.zeros(len(b.kv_lens), b.hkv, 96, dtype=torch.int32, device="cuda")
        lens, _ = api.rpa_evict_kv_cache(x["kv"], x["lens"], x["pages"], x["num"], w, x["budgets"], 96, sinks=2, recent=8,
                                         kv_lens_out=x["lens"], weights_out=w, slots_out=slots, workspace=ws)
        return [q, k, v, out, w, slots, lens, x["kv"]]


def bits(xs):
    return [x.clone().view(torch.uint8) for x in xs]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def alone(step):
    ws = step.workspace()
    step.write()
    torch.cuda.synchronize()
    got = bits(step.run(ws))
    torch.cuda.synchronize()
    assert api.check_device_status(ws) == 0
    return got


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", BATCHES)
def test_inputs_written_late_on_another_stream_than_the_current_one(kind, d):
    step = Step(Batch(*BATCHES[kind], 8, 2, d, 16, seed=d))
    want = alone(step)
    for x in step.dev.values():
        x.zero_()
    ws, stream = step.workspace(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)
        step.write()
        got = bits(step.run(ws))
    stream.synchronize()
    assert api.check_device_status(ws) == 0 and same(got, want)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_two_graphs_that_share_a_workspace(d):
    steps = [Step(Batch(*BATCHES[k], 8, 2, d, 16, seed=d), seed=1) for k in BATCHES]
    want = [alone(s) for s in steps]
    ws = torch.zeros(max(s.bytes for s in steps), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for s in steps:
        s.write()
        s.run(ws)  # (kernels are loaded before a capture)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.write()
            outs.append(s.run(ws))
        graphs.append(graph)
    for i in (0, 1, 1, 0, 0, 1):
        graphs[i].replay()
        torch.cuda.synchronize()
        assert api.check_device_status(ws) == 0 and same(bits(outs[i]), want[i])


def test_steps_on_two_streams():
    steps = [Step(Batch(*BATCHES[k], 8, 2, 128, 16, seed=3), seed=2) for k in BATCHES]
    want = [alone(s) for s in steps]
    streams, spaces = [torch.cuda.Stream() for _ in steps], [s.workspace() for s in steps]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(steps):
            with torch.cuda.stream(streams[i]):
                s.write()
                got[i].append(bits(s.run(spaces[i])))
    torch.cuda.synchronize()
    for i in range(2):
        assert api.check_device_status(spaces[i]) == 0 and all(same(x, want[i]) for x in got[i])
