"""The eviction's parameters on the host: fields that came later, and what they refuse."""
import ctypes

import pytest

from ragged_paged_attention_gb300 import api
from ragged_paged_attention_gb300 import build as rpa_build

FIRST_FORM = 48  # bytes of rpa_evict_params before `positions`


@pytest.fixture(scope="module")
def lib():
    rpa_build.build()
    return api.load_library()


def params(**kw):
    p = api.rpa_evict_params(ctypes.sizeof(api.rpa_evict_params), 1, 2, 512, 8, 16, 2, 4, 32, 1, 3, 0)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def ptrs(n):
    return [ctypes.c_void_p(4096 * (i + 1)) for i in range(n)]


def test_a_struct_without_positions_is_taken_as_before(lib):
    n = ctypes.c_size_t(0)
    assert api.rpa_evict_params.positions.offset == FIRST_FORM
    p = params(struct_size=FIRST_FORM, positions=4096)  # (what lies behind it is not read)
    assert lib.rpa_evict_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0 and n.value > 256
    assert lib.rpa_evict_kv_cache(ctypes.byref(p), *ptrs(9), ctypes.c_void_p(1 << 20), n.value - 1, None) == -8
    p = params(struct_size=FIRST_FORM - 4)
    assert lib.rpa_evict_workspace_size(ctypes.byref(p), ctypes.byref(n)) == -4


def test_positions_alias_nothing(lib):
    n = ctypes.c_size_t(0)
    for i in range(9):
        p = params(positions=4096 * (i + 1))
        assert lib.rpa_evict_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0
        assert lib.rpa_evict_kv_cache(ctypes.byref(p), *ptrs(9), ctypes.c_void_p(1 << 20), n.value, None) == -4
    p = params(positions=4096 * 10)  # (then the workspace is looked at)
    assert lib.rpa_evict_kv_cache(ctypes.byref(p), *ptrs(9), ctypes.c_void_p(1 << 20), n.value - 1, None) == -8


@pytest.mark.parametrize("sizes,code", [(dict(max_num_seqs=32768, num_kv_heads=256, max_keys=38400), -2), (dict(max_num_seqs=32768, num_kv_heads=256, max_keys=32640), 0),
                                        (dict(max_keys=2 ** 31 - 1), 0), (dict(max_num_seqs=128, max_keys=2 ** 31 - 1), -2)], ids=str)
def test_more_blocks_than_a_grid_has_are_refused(lib, sizes, code):
    # a block moves 128 keys of a head: a grid has at most 2^31 - 1 of them
    p, n = params(**sizes), ctypes.c_size_t(0)
    assert lib.rpa_evict_workspace_size(ctypes.byref(p), ctypes.byref(n)) == code
