"""Batches and plain float64 forms for the 4-bit cache, the key weights and the eviction, on CPU tensors."""
import math

import numpy as np
import torch

BF16 = torch.bfloat16


def group_of(d):
    return 32 if d == 64 else 64


def row_bytes(d):
    return d + 8 * (d // group_of(d))


def pack_rows(k, v):
    """bf16 k, v [..., d] -> rows uint8 [..., row_bytes], as include/rpa.h defines them (float32 arithmetic, which
    has the definition's roundings: differences of bf16 values, one division each)."""
    d = k.shape[-1]
    numbers, params = [], []
    for x in (k, v):
        x = torch.where(x.isnan(), torch.zeros_like(x), x).float().clamp(-2.0 ** 48, 2.0 ** 48)
        x = x.unflatten(-1, (-1, group_of(d)))
        m = x.amin(-1, keepdim=True)
        s = ((x.amax(-1, keepdim=True) - m) / 15.0).to(BF16)
        n = torch.where(s > 0, torch.round((x - m) / s.float()), torch.zeros_like(x)).clamp(max=15).to(torch.uint8).flatten(-2)
        numbers.append(n[..., 0::2] + 16 * n[..., 1::2])
        params.append(torch.cat([s, m.to(BF16)], -1).flatten(-2).view(torch.uint8))
    return torch.cat(numbers + params, -1)


def unpack_rows(rows, d):
    """rows -> k, v [..., d] float64, exactly."""
    n = d // group_of(d)
    x = torch.stack([rows[..., :d] & 15, rows[..., :d] >> 4], -1).flatten(-2).double()
    sm = rows[..., d:].contiguous().view(BF16).double().unflatten(-1, (2 * n, 2))
    x = x.unflatten(-1, (2 * n, -1)) * sm[..., :1] + sm[..., 1:]
    return x[..., :n, :].flatten(-2), x[..., n:, :].flatten(-2)


class Batch:
    """A ragged batch over a paged cache. What must not be read is poisoned: NaN in the slots past a sequence's keys (and
    in unused pages), page ids past the sequence, rows and metadata behind the last one."""

    def __init__(self, q_lens, kv_lens, hq, hkv, d, ps, *, g4=True, dtype=BF16, seed=0, pad=2, slots=1, spare=2):
        g = torch.Generator().manual_seed(seed)
        n = len(q_lens)
        self.q_lens, self.lens, self.hq, self.hkv, self.d, self.ps, self.g4 = list(q_lens), list(kv_lens), hq, hkv, d, ps, g4
        self.t = sum(q_lens)
        pps = max(1, -(-max(kv_lens) // ps)) + 1
        count = [-(-k // ps) for k in kv_lens]
        total = sum(count) + spare
        perm = torch.randperm(total, generator=g).to(torch.int32)
        self.table = torch.full((n + slots, pps), 2 ** 31 - 1, dtype=torch.int32)
        at = 0
        for i, c in enumerate(count):
            self.table[i, :c] = perm[at:at + c]
            at += c
        k, v = (torch.randn(total, ps, hkv, d, generator=g).to(BF16) for _ in range(2))
        self.used = torch.zeros(total * ps, dtype=torch.bool)
        self.place = []  # each sequence's slots
        for i, m in enumerate(kv_lens):
            self.place.append((self.table[i, :count[i], None].long() * ps + torch.arange(ps)).flatten()[:m])
            self.used[self.place[-1]] = True
        if g4:
            kv = pack_rows(k, v)
            flat = kv.view(total * ps, hkv, -1)
            flat[~self.used] = 255  # (numbers 15, s and m NaN)
        else:
            kv = torch.stack([k, v], 3).view(total, ps, 2 * hkv, d)
            kv.view(total * ps, 2 * hkv, d)[~self.used] = math.nan
            kv = kv.to(dtype) if dtype.is_floating_point else kv.nan_to_num(0.0).float().mul(20).to(dtype)
        self.kv = kv
        self.kv_lens = torch.tensor(list(kv_lens) + [-7] * slots, dtype=torch.int32)
        self.cu = torch.tensor([0] + np.cumsum(q_lens).tolist() + [10 ** 9] * slots, dtype=torch.int32)
        self.num = torch.tensor([n], dtype=torch.int32)
        self.q = torch.randn(self.t + pad, hq, d, generator=g).to(BF16)
        self.q[self.t:] = math.nan
        self.total = total

    def gpu(self):
        """(kv, kv_lens, page table, cu_q_lens, num_seqs) on the GPU."""
        return tuple(x.cuda() for x in (self.kv, self.kv_lens, self.table, self.cu, self.num))

    def values(self, i):
        """K and V [keys, hkv, d] of sequence i in float64."""
        rows = self.kv.view(torch.uint8).flatten(0, 1)[self.place[i]].contiguous()
        if self.g4:
            return unpack_rows(rows, self.d)
        x = rows.view(self.kv.dtype).double()
        return x[:, 0::2], x[:, 1::2]

    def probabilities(self, i, sm_scale, window=None, cap=None):
        """softmax [hq, q, keys] of sequence i, float64."""
        a, n, k = int(self.cu[i]), self.q_lens[i], self.lens[i]
        keys, _ = self.values(i)
        w = torch.einsum("qhd,khd->hqk", self.q[a:a + n].double(), keys.repeat_interleave(self.hq // self.hkv, 1)) * sm_scale
        if cap:
            w = cap * torch.tanh(w / cap)
        at, key = torch.arange(k - n, k)[:, None], torch.arange(k)[None]
        hidden = key > at
        if window:
            hidden = hidden | (key <= at - window)
        return torch.softmax(w.masked_fill(hidden, -math.inf), -1)

    def attention(self, sm_scale, window=None, cap=None):
        """[tokens, hq, d] float64."""
        out = torch.zeros(self.t, self.hq, self.d, dtype=torch.float64)
        for i, n in enumerate(self.q_lens):
            if n:
                a = int(self.cu[i])
                v = self.values(i)[1].repeat_interleave(self.hq // self.hkv, 1)
                out[a:a + n] = torch.einsum("hqk,khd->qhd", self.probabilities(i, sm_scale, window, cap), v)
        return out
