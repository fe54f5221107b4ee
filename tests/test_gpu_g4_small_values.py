"""Attention over 4-bit caches whose V has scales about 2^-9, where long queries go from f16 to bf16, against float64."""
import math

import pytest
import torch

from long_context import BF16, Batch, group_of, unpack_rows
from ragged_paged_attention_gb300 import api

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -9  # the least scale that f16 takes where |m| < 2^-6
# scales and minima of the groups, from a uniform number: any group's own
SCALES = {"tiny": lambda u: 2.0 ** -12 * (1 + u), "below": lambda u: STEP * (0.6 + 0.39 * u), "at": lambda u: torch.full_like(u, STEP),
          "above": lambda u: STEP * (1 + 0.5 * u), "twice": lambda u: STEP * (2 + u), "either side": lambda u: STEP * (0.7 + 0.6 * u)}
LEAST = {"centre": lambda s, u: s * (u - 8), "near 0": lambda s, u: s * (u - 0.5), "inside": lambda s, u: s * (u - 2.8),
         "about 2^-6": lambda s, u: 2.0 ** -6 * (0.8 + 0.4 * u), "past 2^-6": lambda s, u: -2.0 ** -6 * (1 + u)}


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("m", LEAST)
@pytest.mark.parametrize("s", SCALES)
def test_small_values_of_v(s, m, d):
    b = Batch([300, 1, 40, 150], [900, 700, 40, 600], 8, 2, d, 16, seed=d)
    n = d // group_of(d)
    p = b.kv[..., d:].contiguous().view(BF16).unflatten(-1, (2, 2 * n))
    used = b.used.view(b.total, b.ps)
    u = torch.rand(2, *p[:, :, :, 1, 0::2].shape, generator=torch.Generator().manual_seed(d))
    step = SCALES[s](u[0])
    for j, x in enumerate((step, LEAST[m](step, u[1]))):
        p[:, :, :, 1, j::2][used] = x[used].to(BF16)
    b.kv[..., d:] = p.flatten(-2).view(torch.uint8)
    kv, lens, pages, cu, num = b.gpu()
    ws = torch.zeros(api.rpa_g4_workspace_size(api.make_g4_params(b.q.cuda(), kv, pages)), dtype=torch.uint8, device="cuda")
    got = api.rpa_g4_forward(b.q.cuda(), kv, lens, pages, cu, num, sm_scale=d ** -0.5, workspace=ws)[:b.t].double().cpu()
    assert api.check_device_status(ws) == 0
    want = b.attention(d ** -0.5)
    # Independent roundings of the output, P and K, each 2^-8 of a value at most and 2^-8 / sqrt(3) in the root mean square (a
    # score moves by K's at unit q and k, sm_scale sqrt(d) of it). V's: in bf16 as much again; in f16 at most 2^-15 and
    # 2^-15 again for m, each over sqrt(3) in the root mean square, beside V's own (outputs of long averages are smaller,
    # and so are the errors)
    values = unpack_rows(b.kv.flatten(0, 1)[b.used], d)[1]
    one = 2.0 ** -8 / math.sqrt(3)
    v = max(one, math.sqrt(2) * 2.0 ** -15 / math.sqrt(3) / float(values.pow(2).mean().sqrt()))
    tol = math.sqrt(3 * one ** 2 + v ** 2)
    err, norm = (got - want).norm(), want.norm()
    assert err <= tol * norm, (float(err / norm), tol)
    # the largest of up to 2^21 of them within 6 of their deviations, on values of the greatest's size
    assert (got - want).abs().max() <= 6 * tol * values.abs().max()
