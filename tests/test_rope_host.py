"""Rotary positions and the appending calls without a GPU: the table against the formulas, and what
the calls refuse before they launch anything."""
import ctypes
import math

import pytest
import torch

import plain
from ragged_paged_attention_gb300 import api
from ragged_paged_attention_gb300 import build as rpa_build

LLAMA3 = {"type": "llama3", "factor": 8.0, "low_freq_factor": 1.0, "high_freq_factor": 4.0,
          "original_max_position": 8192}
YARN = {"type": "yarn", "factor": 40.0, "original_max_position": 4096}


@pytest.fixture(scope="module")
def lib():
    rpa_build.build()
    return api.load_library()


@pytest.mark.parametrize("rot", [2, 6, 64, 128, 256])
@pytest.mark.parametrize("base,scaling", [
    (10000.0, None), (500000.0, LLAMA3), (10000.0, YARN), (10000.0, {"type": "linear", "factor": 4.0}),
    (1000.0, {"type": "ntk", "factor": 3.0}), (10000.0, {**YARN, "attention_factor": 1.0}),
    (10000.0, {**YARN, "beta_fast": 3.0, "beta_slow": 2.9}), (1.5, None)])
def test_table_follows_the_formulas(lib, rot, base, scaling):
    if rot == 2 and scaling and scaling["type"] == "ntk":
        pytest.skip("NTK's exponent needs more than one pair")
    t = api.make_rope_table(rot, base=base, scaling=scaling)
    f, amp = plain.frequencies(rot, base, scaling)
    turns = torch.tensor([t.step[i] / 2.0 ** 64 for i in range(rot // 2)], dtype=torch.float64)
    # float64 on both sides: a power, two products and a quotient, and a step of 2^-64
    assert ((turns * 2 * math.pi - f).abs() <= f * 2.0 ** -48 + 2.0 ** -60).all()
    assert t.amplitude == pytest.approx(amp, rel=2.0 ** -24)
    assert all(t.step[i] == 0 for i in range(rot // 2, 128))


def params(**over):
    p = api.rope_params(struct_size=ctypes.sizeof(api.rope_params), version=1, rotary_dim=64, pairing=0, scaling=0,
                        base=10000.0)
    for k, v in over.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("over,code", [
    (dict(rotary_dim=63), -2), (dict(rotary_dim=258), -2), (dict(rotary_dim=-2), -2), (dict(pairing=2), -4),
    (dict(scaling=5), -4), (dict(scaling=-1), -4), (dict(base=1.0), -4), (dict(base=math.nan), -4),
    (dict(base=math.inf), -4), (dict(scaling=1, factor=0.5), -4), (dict(scaling=1, factor=math.nan), -4),
    (dict(scaling=2, factor=2.0, rotary_dim=2), -2), (dict(scaling=3, factor=8.0), -4),
    (dict(scaling=3, factor=8.0, original_max_position=8192, low_freq_factor=4.0, high_freq_factor=4.0), -4),
    (dict(scaling=4, factor=8.0, original_max_position=4096, beta_fast=1.0, beta_slow=1.0), -4),
    (dict(scaling=4, factor=8.0, original_max_position=0, beta_fast=32.0, beta_slow=1.0), -4),
    (dict(attention_factor=-1.0), -4), (dict(attention_factor=1e300), -4), (dict(version=2), -4),
    (dict(struct_size=8), -4), (dict(rotary_dim=0), 0), (dict(attention_factor=0.5), 0)])
def test_table_refusals(lib, over, code):
    p, t = params(**over), api.rope_table()
    assert lib.rope_table_init(ctypes.byref(p), ctypes.byref(t)) == code
    if code:
        assert lib.rpa_last_error()
    assert lib.rope_table_init(None, ctypes.byref(t)) == -1


def test_scaling_names_are_checked(lib):
    for bad in ({"type": "none", "factor": 2.0}, {"type": "linear"}, {"type": "dynamic", "factor": 2.0}, {"factor": 2.0},
                {"type": "llama3", "factor": 8.0}):
        with pytest.raises(ValueError):
            api.make_rope_table(64, scaling=bad)


def apply_params(**over):
    p = api.rope_apply_params(struct_size=ctypes.sizeof(api.rope_apply_params), version=1, num_tokens=5, num_q_heads=4,
                              num_k_heads=2, head_dim=64)
    for k, v in over.items():
        setattr(p, k, v)
    return p


# (num_tokens 5: q is 5 x 4 x 64 elements = 2560 bytes, k half of it)
Q, K, POS, QO, KO = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000


@pytest.mark.parametrize("over,ptrs,code", [
    (dict(num_tokens=-1), {}, -2), (dict(num_q_heads=0), {}, -2), (dict(head_dim=72), {}, -5), (dict(head_dim=528), {}, -5),
    (dict(head_dim=48), {}, -2), (dict(inverse=2), {}, -4), (dict(version=9), {}, -4), (dict(struct_size=16), {}, -4),
    ({}, dict(q=None), -1), ({}, dict(positions=None), -1), ({}, dict(q_out=None), -1), ({}, dict(k=None), -1),
    ({}, dict(k_out=None), -1), (dict(num_k_heads=0), {}, -1), ({}, dict(q=Q + 8), -4), ({}, dict(k_out=KO + 2), -4),
    (dict(q_token_stride=260), {}, -2), (dict(q_head_stride=-64), {}, -2), (dict(q_token_stride=1 << 31), {}, -2),
    (dict(q_out_head_stride=56), {}, -2), (dict(q_out_token_stride=248), {}, -2), (dict(k_out_token_stride=64), {}, -2),
    ({}, dict(q_out=Q + 128), -4), ({}, dict(k_out=K + 512), -4), ({}, dict(q_out=K), -4), ({}, dict(k_out=Q + 512), -4),
    ({}, dict(k_out=QO), -4), (dict(q_out_token_stride=512), dict(q_out=Q), -4)])
def test_apply_refusals(lib, over, ptrs, code):
    t = api.make_rope_table(64)
    at = dict(q=Q, k=K, positions=POS, q_out=QO, k_out=KO, **{})
    at.update(ptrs)
    args = [None if at[n] is None else ctypes.c_void_p(at[n]) for n in ("q", "k", "positions", "q_out", "k_out")]
    p = apply_params(**over)
    assert lib.rope_apply(ctypes.byref(p), ctypes.byref(t), *args, None) == code
    assert lib.rpa_last_error()


def test_apply_table_is_checked_and_no_tokens_launch_nothing(lib):
    args = [ctypes.c_void_p(x) for x in (Q, K, POS, QO, KO)]
    p = apply_params()
    for field, value, code in (("rotary_dim", 66, -2), ("rotary_dim", 7, -2), ("pairing", 3, -4), ("amplitude", math.inf, -4),
                               ("version", 0, -4), ("struct_size", 100, -4)):
        t = api.make_rope_table(64)
        setattr(t, field, value)
        assert lib.rope_apply(ctypes.byref(p), ctypes.byref(t), *args, None) == code, field
    assert lib.rope_apply(ctypes.byref(p), None, *args, None) == -1
    t = api.make_rope_table(64)
    p.num_tokens = 0
    before = lib.rpa_launch_count()
    assert lib.rope_apply(ctypes.byref(p), ctypes.byref(t), *args, None) == 0
    assert lib.rpa_launch_count() == before


def test_apply_accepts_slices_of_one_projection_in_place(lib):
    # q and k as slices of rows of 6 heads, turned in place: the same rows share no element. The call
    # passes every check; num_tokens 0 keeps it from launching, so the layouts are checked by 1 token.
    t = api.make_rope_table(64)
    row = 6 * 64
    p = apply_params(num_tokens=0, q_token_stride=row, k_token_stride=row, q_out_token_stride=row, k_out_token_stride=row)
    q, k = ctypes.c_void_p(Q), ctypes.c_void_p(Q + 4 * 64 * 2)
    assert lib.rope_apply(ctypes.byref(p), ctypes.byref(t), q, k, ctypes.c_void_p(POS), q, k, None) == 0
    # k's slice one head earlier shares q's last head
    p.num_tokens = 3
    k = ctypes.c_void_p(Q + 3 * 64 * 2)
    assert lib.rope_apply(ctypes.byref(p), ctypes.byref(t), q, k, ctypes.c_void_p(POS), q, k, None) == -4


def good_rpa(**over):
    p = api.rpa_params(struct_size=ctypes.sizeof(api.rpa_params), version=1, max_num_tokens=16, num_q_heads=8,
                       num_combined_kv_heads=4, head_dim=128, total_num_pages=8, page_size=16, max_num_seqs=2,
                       pages_per_seq=4, q_dtype=1, kv_dtype=1, sm_scale=1.0, mask_value=math.nan)
    for k, v in over.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("over,rot,strides,ptrs,code", [
    (dict(head_dim=80), 64, {}, {}, -5), (dict(kv_dtype=3), 64, {}, {}, -3), (dict(num_q_heads=5), 64, {}, {}, -2),
    (dict(head_dim=64), 128, {}, {}, -2), (dict(kv_dtype=5), 66, {}, {}, -5), (dict(k_scale=math.nan), 64, {}, {}, -4),
    (dict(k_scale=1e-40), 64, {}, {}, -4), (dict(v_scale=1e-40), 64, {}, {}, -4), ({}, 64, dict(k_token=12), {}, -2),
    ({}, 64, dict(version=0), {}, -4), ({}, 64, dict(struct_size=8), {}, -4), ({}, 64, dict(v_head=-128), {}, -2),
    ({}, 64, {}, dict(new_k=None), -1), ({}, 64, {}, dict(kv_pages=None), -1), ({}, 64, {}, dict(q=None), -1),
    ({}, 64, {}, dict(q_out=None), -1), ({}, 64, {}, dict(new_v=0x200008), -4), ({}, 64, {}, dict(kv_pages=0x400004), -4),
    ({}, 64, {}, dict(q_out=0x100010), -4), ({}, 64, {}, dict(q_out=0x200000), -4), ({}, 64, {}, dict(q_out=0x400000), -4),
    ({}, 64, {}, dict(kv_pages=0x200000), -4)])
def test_update_refusals(lib, over, rot, strides, ptrs, code):
    t = api.make_rope_table(rot)
    at = dict(q=0x100000, new_k=0x200000, new_v=0x300000, kv_pages=0x400000, kv_lens=0x500000, page_indices=0x510000,
              cu=0x520000, num=0x530000, positions=None, q_out=0x600000)
    at.update(ptrs)
    st = api.rope_strides(struct_size=ctypes.sizeof(api.rope_strides), version=1)
    for k, v in strides.items():
        setattr(st, k, v)
    p = good_rpa(**over)
    rc = lib.rpa_rope_update_kv_cache(ctypes.byref(p), ctypes.byref(t), ctypes.byref(st),
                                      *(None if v is None else ctypes.c_void_p(v) for v in at.values()), None, 0, None)
    assert rc == code
    assert lib.rpa_last_error()


def test_update_refuses_a_small_workspace(lib):
    t, p = api.make_rope_table(64), good_rpa()
    ptrs = [ctypes.c_void_p(0x100000 * (i + 1)) for i in range(10)]
    assert lib.rpa_rope_update_kv_cache(ctypes.byref(p), ctypes.byref(t), None, *ptrs, ctypes.c_void_p(256), 64, None) == -8


def test_binding_refuses_cpu_tensors_and_other_tables(lib):
    t = api.make_rope_table(64)
    x, i = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        api.rope_apply(x, None, i, t)
    with pytest.raises(ValueError, match="make_rope_table"):
        api.rope_apply(x, None, i, None)
    with pytest.raises(ValueError, match="CUDA"):
        api.rpa_rope_update_kv_cache(x, x, x, x, i, i, i, i, t)
