"""The 4-bit cache, key weights and eviction on the host: what the entry points and the binding refuse, sizes, and the
definition's own packing."""
import ctypes
import math

import pytest
import torch

from long_context import BF16, group_of, pack_rows, row_bytes, unpack_rows
from ragged_paged_attention_gb300 import api
from ragged_paged_attention_gb300 import build as rpa_build


@pytest.fixture(scope="module")
def lib():
    rpa_build.build()
    return api.load_library()


def g4_params(**kw):
    p = api.rpa_params(struct_size=ctypes.sizeof(api.rpa_params), version=1, max_num_tokens=16, num_q_heads=8,
                       num_combined_kv_heads=4, head_dim=128, total_num_pages=8, page_size=16, max_num_seqs=2, pages_per_seq=4,
                       q_dtype=1, kv_dtype=api.G4, sm_scale=0.1, mask_value=math.nan)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def ptrs(n):
    return [ctypes.c_void_p(4096 * (i + 1)) for i in range(n)]


BAD = [("num_combined_kv_heads", 3, -2), ("num_q_heads", 5, -2), ("head_dim", 96, -5), ("head_dim", 80, -5), ("q_dtype", 2, -3),
       ("kv_dtype", 5, -3), ("sliding_window", -1, -4), ("soft_cap", math.inf, -4), ("mask_value", -1.0, -4), ("k_scale", 1.0, -4),
       ("v_scale", 0.5, -4), ("version", 7, -4), ("struct_size", 4, -4), ("page_size", 0, -2), ("sm_scale", math.nan, -4),
       ("batch_kind", 3, -4)]


@pytest.mark.parametrize("field,value,code", BAD)
def test_g4_calls_refuse(lib, field, value, code):
    p, n = g4_params(**{field: value}), ctypes.c_size_t(0)
    assert lib.rpa_g4_workspace_size(ctypes.byref(p), ctypes.byref(n)) == code
    assert lib.rpa_g4_forward(ctypes.byref(p), *ptrs(7), ctypes.c_void_p(256), 1 << 30, None) == code
    assert lib.rpa_g4_read_kv_cache(ctypes.byref(p), *ptrs(7), None, 0, None) == code
    t = api.make_rope_table(64)
    assert lib.rpa_g4_update_kv_cache(ctypes.byref(p), ctypes.byref(t), None, *ptrs(8), None, ctypes.c_void_p(1 << 20), None, 0, None) == code
    assert lib.rpa_last_error()


def test_g4_calls_refuse_pointers_and_workspaces(lib):
    p, n = g4_params(), ctypes.c_size_t(0)
    assert lib.rpa_g4_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0 and n.value > 256
    assert lib.rpa_g4_workspace_size(ctypes.byref(p), None) == -1
    assert lib.rpa_g4_workspace_size(None, ctypes.byref(n)) == -1
    a, ws = ptrs(7), ctypes.c_void_p(1 << 20)
    for i in range(7):
        assert lib.rpa_g4_forward(ctypes.byref(p), *a[:i], None, *a[i + 1:], ws, n.value, None) == -1
        assert lib.rpa_g4_read_kv_cache(ctypes.byref(p), *a[:i], None, *a[i + 1:], None, 0, None) == -1
    odd = ctypes.c_void_p(4104)
    assert lib.rpa_g4_forward(ctypes.byref(p), odd, *a[1:], ws, n.value, None) == -4
    assert lib.rpa_g4_read_kv_cache(ctypes.byref(p), odd, *a[1:], None, 0, None) == -4
    assert lib.rpa_g4_read_kv_cache(ctypes.byref(p), *a[:6], a[5], None, 0, None) == -4  # k_out is v_out
    assert lib.rpa_g4_read_kv_cache(ctypes.byref(p), *a[:6], a[0], None, 0, None) == -4
    assert lib.rpa_g4_read_kv_cache(ctypes.byref(p), *a, ws, 64, None) == -8
    assert lib.rpa_g4_forward(ctypes.byref(p), *a[:6], a[0], ws, n.value, None) == -4  # out is q
    assert lib.rpa_g4_forward(ctypes.byref(p), *a, ws, n.value - 1, None) == -8
    assert lib.rpa_g4_forward(ctypes.byref(p), *a, None, n.value, None) == -8
    for rot in (8, 24, 72):
        t = api.make_rope_table(rot)
        assert lib.rpa_g4_update_kv_cache(ctypes.byref(p), ctypes.byref(t), None, *ptrs(8), None, ctypes.c_void_p(1 << 20), None, 0, None) == -5


def test_other_calls_take_no_g4_cache(lib):
    p, n = g4_params(), ctypes.c_size_t(0)
    assert lib.rpa_workspace_size(ctypes.byref(p), ctypes.byref(n)) == -3
    assert lib.rpa_cross_workspace_size(ctypes.byref(p), ctypes.byref(n)) == -3
    assert lib.rpa_forward(ctypes.byref(p), *ptrs(7), ctypes.c_void_p(256), 1 << 30, None) == -3
    assert lib.rpa_update_kv_cache(ctypes.byref(p), *ptrs(7), None, 0, None) == -3


@pytest.mark.parametrize("field,value,code", [x for x in BAD if x[0] != "kv_dtype"] + [("kv_dtype", 2, -3), ("kv_dtype", 5, -3)])
def test_key_weights_refuse(lib, field, value, code):
    p, n = g4_params(**{field: value}), ctypes.c_size_t(0)
    assert lib.rpa_key_weights_workspace_size(ctypes.byref(p), ctypes.byref(n)) == code
    assert lib.rpa_key_weights(ctypes.byref(p), *ptrs(8), 1.0, ctypes.c_void_p(256), 1 << 30, None) == code


def test_key_weights_refuse_pointers_and_workspaces(lib):
    for kind in (api.G4, api.BF16):
        p, n = g4_params(kv_dtype=kind), ctypes.c_size_t(0)
        assert lib.rpa_key_weights_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0 and n.value > 256
        a, ws = ptrs(8), ctypes.c_void_p(1 << 20)
        for i in range(8):
            assert lib.rpa_key_weights(ctypes.byref(p), *a[:i], None, *a[i + 1:], 1.0, ws, n.value, None) == -1
        assert lib.rpa_key_weights(ctypes.byref(p), *a, math.inf, ws, n.value, None) == -4
        assert lib.rpa_key_weights(ctypes.byref(p), *a, math.nan, ws, n.value, None) == -4
        assert lib.rpa_key_weights(ctypes.byref(p), *a[:7], a[0], 1.0, ws, n.value, None) == -4
        assert lib.rpa_key_weights(ctypes.byref(p), *a, 1.0, ws, n.value - 1, None) == -8
    p = g4_params(kv_dtype=api.BF16, head_dim=96)
    assert lib.rpa_key_weights_workspace_size(ctypes.byref(p), ctypes.byref(n)) == -5


def evict_params(**kw):
    p = api.rpa_evict_params(ctypes.sizeof(api.rpa_evict_params), 1, 2, 512, 8, 16, 2, 4, 32, 1, 3, 0)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("field,value,code", [("num_kv_heads", 0, -2), ("row_bytes", 0, -2), ("row_bytes", 40, -2), ("total_num_pages", 0, -2),
                                              ("page_size", 0, -2), ("max_num_seqs", 0, -2), ("pages_per_seq", 0, -2), ("max_keys", 0, -2),
                                              ("max_keys", 3, -4), ("sinks", -1, -4), ("recent", -1, -4), ("recent", 2 ** 31 - 1, -4),
                                              ("version", 9, -4), ("struct_size", 8, -4), ("pages_per_seq", 2 ** 31 - 1, -2)])
def test_evict_refuses(lib, field, value, code):
    p, n = evict_params(**{field: value}), ctypes.c_size_t(0)
    assert lib.rpa_evict_workspace_size(ctypes.byref(p), ctypes.byref(n)) == code
    assert lib.rpa_evict_kv_cache(ctypes.byref(p), *ptrs(9), ctypes.c_void_p(256), 1 << 30, None) == code


def test_evict_refuses_pointers_and_workspaces(lib):
    p, n = evict_params(), ctypes.c_size_t(0)
    assert lib.rpa_evict_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0 and n.value > 256
    a, ws = ptrs(9), ctypes.c_void_p(1 << 20)
    for i in (0, 1, 2, 3, 4, 5, 7):
        assert lib.rpa_evict_kv_cache(ctypes.byref(p), *a[:i], None, *a[i + 1:], ws, n.value, None) == -1
    assert lib.rpa_evict_kv_cache(ctypes.byref(p), ctypes.c_void_p(4104), *a[1:], ws, n.value, None) == -4
    assert lib.rpa_evict_kv_cache(ctypes.byref(p), *a[:7], a[1], a[8], ws, n.value, None) == -4  # slots_out is kv_lens
    assert lib.rpa_evict_kv_cache(ctypes.byref(p), *a[:6], a[5], *a[7:], ws, n.value, None) == -4  # kv_lens_out is budgets
    assert lib.rpa_evict_kv_cache(ctypes.byref(p), *a, ws, n.value - 1, None) == -8
    assert lib.rpa_evict_kv_cache(None, *a, ws, n.value, None) == -1


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows(d):
    assert api.g4_row_bytes(d) == row_bytes(d) and row_bytes(d) % 16 == 0
    k, v = (torch.randn(5, 3, d, generator=torch.Generator().manual_seed(i)).to(BF16) for i in range(2))
    rows = pack_rows(k, v)
    assert rows.shape == (5, 3, row_bytes(d))
    for x, y in zip((k, v), unpack_rows(rows, d)):
        g = x.double().unflatten(-1, (-1, group_of(d)))
        s = (g.amax(-1) - g.amin(-1)) / 15 * (1 + 2.0 ** -8)
        assert ((x.double() - y).abs() <= s.repeat_interleave(group_of(d), -1) / 2).all()
        assert torch.equal(y.unflatten(-1, (-1, group_of(d))).amin(-1), g.amin(-1))
    with pytest.raises(ValueError):
        api.g4_row_bytes(96)


def test_binding_refuses_cpu_tensors():
    x, i = torch.zeros(4, 4, 128, dtype=BF16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        api.rpa_g4_forward(x, x, i, i, i, i)
    with pytest.raises(ValueError):
        api.rpa_g4_update_kv_cache(x, x, x, x, i, i, i, i, api.rope_table())
    with pytest.raises(ValueError):
        api.rpa_g4_read_kv_cache(x, i, i, i, i, 4)
    with pytest.raises(ValueError):
        api.rpa_key_weights(x, x, i, i, i, i, x)
    with pytest.raises(ValueError):
        api.rpa_evict_kv_cache(x, i, i, i, x, i, 4)
