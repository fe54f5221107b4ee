"""Host-side checks of the appending and rotating calls that need no GPU: what they refuse before they
launch anything, and layouts that they must let through."""
import ctypes
import math

import pytest

from ragged_paged_attention_gb300 import api
from ragged_paged_attention_gb300 import build as rpa_build


@pytest.fixture(scope="module")
def lib():
    rpa_build.build()
    return api.load_library()


def at(*addresses):
    return [None if x is None else ctypes.c_void_p(x) for x in addresses]


def rpa(**over):
    p = api.rpa_params(struct_size=ctypes.sizeof(api.rpa_params), version=1, max_num_tokens=16, num_q_heads=8,
                       num_combined_kv_heads=4, head_dim=128, total_num_pages=8, page_size=16, max_num_seqs=2,
                       pages_per_seq=4, q_dtype=1, kv_dtype=1, sm_scale=1.0, mask_value=math.nan)
    for k, v in over.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("offset", [1, 2, 3, 255])
def test_cache_writes_refuse_a_workspace_whose_error_word_is_misaligned(lib, offset):
    # an atomic on a misaligned word faults: refused, whatever else the workspace is used for
    ws, p = ctypes.c_void_p((1 << 24) + offset), rpa()
    m = api.mla_params(struct_size=ctypes.sizeof(api.mla_params), version=1, max_num_tokens=8, num_q_heads=128,
                       lkv_dim=512, r_dim=64, lkv_dim_pad=512, r_dim_pad=128, total_num_pages=4, page_size=64,
                       kv_packing=2, max_num_seqs=2, pages_per_seq=2, sm_scale=0.07, mask_value=math.nan)
    ptrs = at(*(0x100000 * (i + 1) for i in range(11)))
    t = api.make_rope_table(64)
    assert lib.rpa_rope_update_kv_cache(ctypes.byref(p), ctypes.byref(t), None, *ptrs[:8], None, ptrs[9], ws, 512, None) == -8
    assert lib.rpa_update_kv_cache(ctypes.byref(p), *ptrs[:7], ws, 512, None) == -8
    assert lib.mla_update_kv_cache(ctypes.byref(m), *ptrs[:8], ws, 512, None) == -8
    assert lib.rpa_selftest_bounded_wait(ws, 512, None) == -8


# ------------------------------------------------------------------ operands between one another
NO_GPU = -6  # every check passed: there is no device to launch on


def rows(base, tokens, heads, dim, token, head):
    """Every byte address of an operand's bf16 rows."""
    return {base + 2 * (t * token + h * head) + 2 * e for t in range(tokens) for h in range(heads) for e in range(dim)}


def apply_rc(lib, T, hq, hk, d, q, k, q_out=None, k_out=None):
    """The status of rope_apply on operands given as (address, token stride, head stride)."""
    q_out, k_out = q_out or q, k_out or k
    p = api.rope_apply_params(struct_size=ctypes.sizeof(api.rope_apply_params), version=1, num_tokens=T, num_q_heads=hq,
                              num_k_heads=hk, head_dim=d, q_token_stride=q[1], q_head_stride=q[2], k_token_stride=k[1],
                              k_head_stride=k[2], q_out_token_stride=q_out[1], q_out_head_stride=q_out[2],
                              k_out_token_stride=k_out[1], k_out_head_stride=k_out[2])
    t = api.make_rope_table(16)
    return lib.rope_apply(ctypes.byref(p), ctypes.byref(t), *at(q[0], k[0], 1 << 30, q_out[0], k_out[0]), None)


needs_no_gpu = pytest.mark.skipif("__import__('torch').cuda.is_available()", reason="the addresses are made up")


@needs_no_gpu
@pytest.mark.parametrize("T", [1, 2, 5])
@pytest.mark.parametrize("H", [1, 3])
def test_parts_of_the_same_heads_are_turned_in_place(lib, T, H):
    # [T, H, 3, D]: q, k and v of a head beside one another
    d, base = 64, 1 << 20
    part = lambda i: (base + 2 * i * d, 3 * H * d, 3 * d)  # noqa: E731
    assert apply_rc(lib, T, H, H, d, part(0), part(1)) == NO_GPU
    assert apply_rc(lib, T, H, H, d, part(2), part(0)) == NO_GPU
    assert apply_rc(lib, T, H, H, d, part(0), part(1), k_out=part(2)) == NO_GPU
    # k eight elements early: it shares them with q
    assert apply_rc(lib, T, H, H, d, part(0), (base + 2 * (d - 8), 3 * H * d, 3 * d)) == -4


@needs_no_gpu
def test_slices_of_one_projection_are_turned_in_place(lib):
    row, d = 6 * 64, 64
    q, k = (1 << 20, row, d), ((1 << 20) + 4 * d * 2, row, d)
    for T in (1, 2, 7):
        assert apply_rc(lib, T, 4, 2, d, q, k) == NO_GPU
        assert apply_rc(lib, T, 4, 2, d, q, (k[0] - 16, row, d)) == -4
    # one head, one token: the strides of such a dimension say nothing
    assert apply_rc(lib, 5, 1, 1, d, (1 << 20, 4 * d, d), ((1 << 20) + 2 * d, 4 * d, 8 * d)) == NO_GPU
    assert apply_rc(lib, 1, 2, 1, d, (1 << 20, 8 * d, d), ((1 << 20) + 4 * d, 2 * d, d)) == NO_GPU
    assert apply_rc(lib, 5, 1, 1, d, (1 << 20, 4 * d, d), (1 << 24, 4 * d, d), q_out=(1 << 20, 4 * d, 2 * d)) == NO_GPU


@needs_no_gpu
def test_overlap_is_told_from_interleaving(lib):
    """Small layouts of equal strides in and out of order, against the sets of addresses themselves."""
    seen = {True: 0, False: 0}
    for d, head, token in ((16, 16, 64), (16, 48, 144), (16, 64, 16), (16, 40, 136), (32, 96, 40), (16, 16, 16), (16, 80, 32)):
        for T, hq, hk in ((1, 1, 1), (3, 2, 2), (2, 3, 1), (4, 1, 2)):
            for shift in range(-20, 21):
                q, k = (1 << 20, token, head), ((1 << 20) + 16 * shift, token, head)
                dense = [(1 << 24, 0, 0), (1 << 25, 0, 0)]
                # k's output between q's rows; q's output is elsewhere
                rc = apply_rc(lib, T, hq, hk, d, q, dense[0], dense[1], k)
                if rc == -2:
                    continue  # (k's rows overlap one another)
                shared = bool(rows(q[0], T, hq, d, token, head) & rows(k[0], T, hk, d, token, head))
                assert rc == (-4 if shared else NO_GPU), (d, head, token, T, hq, hk, shift)
                seen[shared] += 1
    assert min(seen.values()) > 100


def test_a_captured_calls_cached_workspace_outlives_its_replacement(monkeypatch):
    # (rpa_forward's and the others' that share one per device: a graph holds the address)
    import weakref

    import torch
    monkeypatch.setattr(api.Workspace, "_cache", {})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    eager = weakref.ref(api.Workspace.get(300, "cpu", "a"))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    captured = weakref.ref(api.Workspace.get(1000, "cpu", "a"))
    assert eager() is None and captured().numel() == 1000
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    assert api.Workspace.get(5000, "cpu", "a").numel() == 5000
    assert captured() is not None and captured().numel() == 1000
