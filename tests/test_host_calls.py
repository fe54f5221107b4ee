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
