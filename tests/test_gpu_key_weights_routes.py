"""Key weights where the workspace has no room for every sequence's scores."""
import pytest
import torch

from long_context import BF16, Batch, row_bytes
from ragged_paged_attention_gb300 import api
from test_gpu_long_context import LENS, check_weights

pytestmark = pytest.mark.gpu

SCORES = 1 << 27  # floats of scores that the workspace takes at most


def capacity(b):
    """Floats that the scores of every sequence would take at the page table's full width."""
    g, n = b.hq // b.hkv, len(b.kv_lens)
    return b.table.shape[1] * b.ps * b.hkv * min(16 * n, 4 * n + 2 * b.q.shape[0] * g)


def widen(b, to):
    """The batch with a page table whose capacity is past `to`."""
    one = capacity(b) // b.table.shape[1]
    b.table = torch.cat([b.table, torch.full((b.table.shape[0], to // one + 1 - b.table.shape[1]), 2 ** 31 - 1, dtype=torch.int32)], 1)
    assert capacity(b) > to
    return b


@pytest.mark.parametrize("g4", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_lens,kv_lens,kw", [(*LENS, {}), ([1] * 30, list(range(1, 3000, 100)), {}), ([1, 2], [900, 40], {}), ([40, 150], [900, 400], {}),
                                               (*LENS, dict(sliding_window=130)), (*LENS, dict(soft_cap=20.0, keep=0.0)), (*LENS, dict(sm_scale=-0.1))],
                         ids=["mixed", "decodes", "few", "windows", "window", "cap", "negative"])
def test_tables_wider_than_the_room_for_scores(q_lens, kv_lens, kw, d, g4):
    check_weights(widen(Batch(q_lens, kv_lens, 8, 2, d, 16, g4=g4, seed=d), SCORES), **kw)


@pytest.mark.parametrize("g4", [False, True])
@pytest.mark.parametrize("others", [[], [40, 130]], ids=["decodes", "mixed"])
def test_more_scores_than_the_workspace_takes(others, g4):
    # 80 decodes of 16 rows a KV head over 55000 to 60000 keys: more than 2^27 scores, so that the last sequences' are computed again
    hq, hkv, d, ps = 32, 2, 64, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    q_lens, kv_lens = [1] * 80 + others, [55000 + 63 * i for i in range(80)] + [3000 + 7 * n for n in others]
    assert sum(k * hkv * 16 for k in kv_lens[:80]) > SCORES
    count = [-(-k // ps) for k in kv_lens]
    total = sum(count)
    table = torch.full((len(q_lens), max(count)), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    perm = torch.randperm(total, generator=g, device="cuda").int()
    for i, c in enumerate(count):
        table[i, :c] = perm[sum(count[:i]):sum(count[:i]) + c]
    if g4:
        kv = torch.randint(0, 256, (total, ps, hkv, row_bytes(d)), generator=g, device="cuda", dtype=torch.uint8)
        sm = torch.rand(total, ps, hkv, 4, 2, generator=g, device="cuda")
        kv[..., d:] = torch.stack([0.2 + 0.1 * sm[..., 0], -2.0 + 0.5 * sm[..., 1]], -1).to(BF16).flatten(-2).view(torch.uint8)
    else:
        kv = torch.empty(total, ps, 2 * hkv, d, dtype=BF16, device="cuda").normal_(generator=g)
    lens = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + q_lens, device="cuda").cumsum(0).int()
    num = torch.tensor([len(q_lens)], dtype=torch.int32, device="cuda")
    q = torch.randn(sum(q_lens), hq, d, generator=g, device="cuda").to(BF16)
    old = torch.rand(total, hkv, ps, generator=g, device="cuda") * 1e-4
    prm = api._batch_params(q.get_device(), *q.shape, kv, lens, table, cu, num, g4=g4)
    ws = torch.zeros(api.rpa_key_weights_workspace_size(prm), dtype=torch.uint8, device="cuda")
    out = api.rpa_key_weights(q, kv, lens, table, cu, num, old, sm_scale=d ** -0.5, keep=0.5, weights_out=torch.full_like(old, -3.0), workspace=ws)
    assert api.check_device_status(ws) == 0
    # test_gpu_long_context.check_weights' bound, on values of 4-bit rows up to some 2.5 in place of unit ones: sum |q k| is
    # at most 0.8 * 2.5 d
    rel = 2 * (d + 8) * 2.0 ** -24 * 2.0 * d * d ** -0.5 + 2.0 ** -20
    for i, (n, k) in enumerate(zip(q_lens, kv_lens)):
        page = table[i, :count[i]].long()
        rows = kv[page].flatten(0, 1)[:k]
        if g4:
            x = torch.stack([rows[..., :d // 2] & 15, rows[..., :d // 2] >> 4], -1).flatten(-2).double().unflatten(-1, (2, 32))
            p = rows[..., d:d + 8].contiguous().view(BF16).double().unflatten(-1, (2, 2))
            keys = (x * p[..., :1] + p[..., 1:]).flatten(-2)
        else:
            keys = rows[:, 0::2].double()
        a = int(cu[i])
        s = torch.einsum("qhgd,khd->hgqk", q[a:a + n].double().unflatten(1, (hkv, -1)), keys) * d ** -0.5
        hidden = torch.arange(k, device="cuda") > torch.arange(k - n, k, device="cuda")[:, None]
        new = torch.softmax(s.masked_fill(hidden, -torch.inf), -1).sum((1, 2))  # [hkv, keys]
        was, got = (x[page].transpose(1, 2).flatten(0, 1)[:k].T.double() for x in (old, out))
        want = 0.5 * was + new
        assert ((got - want).abs() <= rel * new + 2.0 ** -23 * want).all(), (i, float(((got - want).abs() / want).max()))
        tail = out[page].transpose(1, 2).flatten(0, 1)[k:]
        assert (tail == -3.0).all()
