"""Key weights of pages that sequences share."""
import pytest
import torch

from long_context import Batch
from test_gpu_long_context import weigh

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("g4", [False, True])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 2, 1, 3], [700, 600, 900, 640]), ([40, 150, 1, 64], [700, 650, 900, 640])], ids=["decodes", "windows"])
def test_shared_pages_get_one_sequences_weights(q_lens, kv_lens, g4):
    # out of place: each shared slot holds what one of the sequences gives it, with what it had before added once
    b = Batch(q_lens, kv_lens, 8, 2, 128, 16, g4=g4, seed=6)
    shared = 500 // 16
    for i in range(1, 4):
        b.table[i, :shared] = b.table[0, :shared]
        b.place[i] = torch.cat([b.place[0][:shared * 16], b.place[i][shared * 16:]])
    old, keep, scale = torch.rand(b.total, 2, 16, generator=torch.Generator().manual_seed(1)), 0.75, 128 ** -0.5
    rel = 2 * (128 + 8) * 2.0 ** -24 * 0.64 * 128 * scale + 2.0 ** -20  # (check_weights')
    for _ in range(3):
        got, bits = weigh(b, old, keep, sm_scale=scale)
        assert bits == 0
        near = []
        for i in range(4):
            new = b.probabilities(i, scale).unflatten(0, (2, -1)).sum((1, 2)).T  # [keys, hkv]
            at = b.place[i]
            want = keep * old[at // 16, :, at % 16].double() + new
            near.append((got[at // 16, :, at % 16].double() - want).abs() <= rel * new + 2.0 ** -23 * want)
        for i in range(4):
            assert near[i][shared * 16:].all(), i
        assert torch.stack([x[:shared * 16] for x in near]).any(0).all()
