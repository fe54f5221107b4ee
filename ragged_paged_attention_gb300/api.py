"""Python binding of ``librpa_gb300.so`` (the C ABI in ``include/rpa.h``).

Argument marshalling only: each function checks dtypes/shapes, turns torch CUDA
tensors into pointers and sizes, and calls the C entry point of the same name on
the current torch stream.  Every step of the computation runs in the library's
CUDA kernels; there is no fallback.  When the library or a CUDA device is missing
the calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os
import re
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librpa_gb300.so")
ABI_VERSION = 1

BF16, FP8_E4M3, F32, INT8, INT4 = 1, 2, 3, 4, 5

STATUS = {0: "RPA_OK", -1: "RPA_ERR_NULL", -2: "RPA_ERR_SHAPE", -3: "RPA_ERR_DTYPE", -4: "RPA_ERR_VALUE",
          -5: "RPA_ERR_UNSUPPORTED", -6: "RPA_ERR_CUDA", -7: "RPA_ERR_DEVICE_CHECK", -8: "RPA_ERR_WORKSPACE"}

EXPORTS = ("rpa_workspace_size", "rpa_forward", "rpa_update_kv_cache", "mla_workspace_size",
           "mla_update_kv_cache", "mla_rpa_forward", "sparse_mla_workspace_size", "sparse_mla_forward",
           "rpa_check_device_status", "rpa_last_error", "rpa_version", "rpa_profile_enable",
           "rpa_profile_reset", "rpa_profile_read", "rpa_forward_noalloc", "rpa_launch_count",
           "rpa_forward_update", "sparse_mla_ragged_workspace_size", "sparse_mla_write_and_attend_ragged",
           "rpa_selftest_bounded_wait", "rope_table_init", "rope_apply", "rpa_rope_update_kv_cache",
           "rpa_rope_forward_update", "rpa_cross_workspace_size", "rpa_cross_forward")


class RpaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code


class rpa_kernel_time(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("launches", ctypes.c_int64), ("total_ms", ctypes.c_double)]


class rpa_params(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("version", ctypes.c_uint32),
                ("max_num_tokens", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_combined_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("total_num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_num_seqs", ctypes.c_int32), ("pages_per_seq", ctypes.c_int32),
                ("q_dtype", ctypes.c_int32), ("kv_dtype", ctypes.c_int32), ("sm_scale", ctypes.c_float),
                ("sliding_window", ctypes.c_int32), ("soft_cap", ctypes.c_float), ("mask_value", ctypes.c_float),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float), ("batch_kind", ctypes.c_int32)]


BATCH_MIXED, BATCH_DECODE_ONLY, BATCH_PREFILL_ONLY = 0, 1, 2


class mla_params(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("version", ctypes.c_uint32),
                ("max_num_tokens", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("lkv_dim", ctypes.c_int32), ("r_dim", ctypes.c_int32), ("lkv_dim_pad", ctypes.c_int32),
                ("r_dim_pad", ctypes.c_int32), ("total_num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("kv_packing", ctypes.c_int32), ("max_num_seqs", ctypes.c_int32),
                ("pages_per_seq", ctypes.c_int32), ("sm_scale", ctypes.c_float),
                ("sliding_window", ctypes.c_int32), ("soft_cap", ctypes.c_float), ("mask_value", ctypes.c_float),
                ("q_dtype", ctypes.c_int32), ("q_scale", ctypes.c_float)]


class sparse_params(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("version", ctypes.c_uint32), ("batch", ctypes.c_int32),
                ("num_queries", ctypes.c_int32), ("num_heads", ctypes.c_int32), ("dk", ctypes.c_int32),
                ("dv", ctypes.c_int32), ("row_stride", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("read_block", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("total_num_pages", ctypes.c_int32), ("seq_len", ctypes.c_int32), ("sm_scale", ctypes.c_float)]


class sparse_ragged_params(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("version", ctypes.c_uint32), ("num_tokens", ctypes.c_int32),
                ("num_seqs", ctypes.c_int32), ("num_heads", ctypes.c_int32), ("dv", ctypes.c_int32),
                ("rope", ctypes.c_int32), ("row_stride", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("read_block", ctypes.c_int32), ("page_size", ctypes.c_int32), ("num_page_ids", ctypes.c_int32),
                ("total_num_pages", ctypes.c_int32), ("sm_scale", ctypes.c_float)]


ROPE_HALF, ROPE_INTERLEAVED, ROPE_MAX_DIM = 0, 1, 256
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "llama3": 3, "yarn": 4}


class rope_params(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("version", ctypes.c_uint32), ("rotary_dim", ctypes.c_int32),
                ("pairing", ctypes.c_int32), ("scaling", ctypes.c_int32), ("original_max_position", ctypes.c_int32),
                ("base", ctypes.c_double), ("factor", ctypes.c_double), ("low_freq_factor", ctypes.c_double),
                ("high_freq_factor", ctypes.c_double), ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double),
                ("attention_factor", ctypes.c_double)]


class rope_table(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("version", ctypes.c_uint32), ("rotary_dim", ctypes.c_int32),
                ("pairing", ctypes.c_int32), ("amplitude", ctypes.c_float), ("reserved", ctypes.c_uint32),
                ("step", ctypes.c_uint64 * (ROPE_MAX_DIM // 2))]


class rope_apply_params(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("version", ctypes.c_uint32), ("num_tokens", ctypes.c_int32),
                ("num_q_heads", ctypes.c_int32), ("num_k_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("inverse", ctypes.c_int32), ("reserved", ctypes.c_int32), ("q_token_stride", ctypes.c_int64),
                ("q_head_stride", ctypes.c_int64), ("k_token_stride", ctypes.c_int64),
                ("k_head_stride", ctypes.c_int64), ("q_out_token_stride", ctypes.c_int64),
                ("q_out_head_stride", ctypes.c_int64), ("k_out_token_stride", ctypes.c_int64),
                ("k_out_head_stride", ctypes.c_int64)]


class rope_strides(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("version", ctypes.c_uint32), ("q_token", ctypes.c_int64),
                ("q_head", ctypes.c_int64), ("k_token", ctypes.c_int64), ("k_head", ctypes.c_int64),
                ("v_token", ctypes.c_int64), ("v_head", ctypes.c_int64)]


_lib = None
_lock = threading.Lock()


def load_library(path: str = LIB_PATH):
    """Load the CUDA library (raises when it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with ragged_paged_attention_gb300.build.build()")
        lib = ctypes.CDLL(path)
        P, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        szp = ctypes.POINTER(ctypes.c_size_t)
        lib.rpa_version.restype = ctypes.c_int
        lib.rpa_last_error.restype = ctypes.c_char_p
        lib.rpa_workspace_size.argtypes = [ctypes.POINTER(rpa_params), szp]
        lib.rpa_forward.argtypes = [ctypes.POINTER(rpa_params), P, P, P, P, P, P, P, P, sz, P]
        lib.rpa_forward_noalloc.argtypes = [ctypes.POINTER(rpa_params), P, P, P, P, P, P, P, P]
        lib.rpa_update_kv_cache.argtypes = [ctypes.POINTER(rpa_params), P, P, P, P, P, P, P, P, sz, P]
        lib.rpa_forward_update.argtypes = [ctypes.POINTER(rpa_params), P, P, P, P, P, P, P, P, P, P, sz, P]
        lib.mla_workspace_size.argtypes = [ctypes.POINTER(mla_params), szp]
        lib.mla_update_kv_cache.argtypes = [ctypes.POINTER(mla_params), P, P, P, P, P, P, P, P, P, sz, P]
        lib.mla_rpa_forward.argtypes = [ctypes.POINTER(mla_params), P, P, P, P, P, P, P, P, P, P, P, P, sz, P]
        lib.sparse_mla_workspace_size.argtypes = [ctypes.POINTER(sparse_params), szp]
        lib.sparse_mla_forward.argtypes = [ctypes.POINTER(sparse_params), P, P, P, P, P, P, P, sz, P]
        lib.sparse_mla_ragged_workspace_size.argtypes = [ctypes.POINTER(sparse_ragged_params), szp]
        lib.sparse_mla_write_and_attend_ragged.argtypes = [ctypes.POINTER(sparse_ragged_params)] + [P] * 14 + [sz, P]
        lib.rope_table_init.argtypes = [ctypes.POINTER(rope_params), ctypes.POINTER(rope_table)]
        lib.rope_apply.argtypes = [ctypes.POINTER(rope_apply_params), ctypes.POINTER(rope_table)] + [P] * 6
        lib.rpa_rope_update_kv_cache.argtypes = [ctypes.POINTER(rpa_params), ctypes.POINTER(rope_table),
                                                 ctypes.POINTER(rope_strides)] + [P] * 11 + [sz, P]
        lib.rpa_rope_forward_update.argtypes = [ctypes.POINTER(rpa_params), ctypes.POINTER(rope_table),
                                                ctypes.POINTER(rope_strides)] + [P] * 12 + [sz, P]
        lib.rpa_cross_workspace_size.argtypes = [ctypes.POINTER(rpa_params), szp]
        lib.rpa_cross_forward.argtypes = [ctypes.POINTER(rpa_params), P, P, P, P, P, P, P, P, sz, P]
        lib.rpa_check_device_status.argtypes = [P, ctypes.POINTER(ctypes.c_uint32), P]
        lib.rpa_selftest_bounded_wait.argtypes = [P, sz, P]
        lib.rpa_profile_enable.argtypes = [ctypes.c_int]
        lib.rpa_profile_reset.argtypes = []
        lib.rpa_profile_read.argtypes = [ctypes.POINTER(rpa_kernel_time), ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
        lib.rpa_launch_count.argtypes = []
        lib.rpa_launch_count.restype = ctypes.c_int64
        for name in EXPORTS:
            if name not in ("rpa_last_error",):
                getattr(lib, name).restype = ctypes.c_int
        if lib.rpa_version() != ABI_VERSION:
            raise RuntimeError(f"library ABI {lib.rpa_version()} != binding ABI {ABI_VERSION}")
        _lib = lib
        return lib


def _check(rc: int):
    if rc != 0:
        msg = _lib.rpa_last_error().decode() if _lib is not None else ""
        raise RpaError(rc, msg)


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _dev(t: torch.Tensor, name: str, dtype=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _opt(x, default=0.0):
    return default if x is None else x


class Workspace:
    """A zero-initialised device buffer reused across calls (one per device and purpose).  One that a call was
    captured with stays when a larger one replaces it: the graph holds its address."""

    _cache: dict = {}
    _captured: dict = {}

    @classmethod
    def get(cls, nbytes: int, device, tag: str = "default") -> torch.Tensor:
        key = (str(device), tag)
        buf = cls._cache.get(key)
        if buf is None or buf.numel() < nbytes:
            buf = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
            cls._cache[key] = buf
        if torch.cuda.is_current_stream_capturing():
            cls._captured[buf.data_ptr()] = buf
        return buf


_kept = threading.local()  # .workspaces: this thread's {(device, stream): workspace}; they go with the thread
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
_current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_BF16, _I32 = torch.bfloat16, torch.int32


def _own_workspaces() -> dict:
    try:
        return _kept.workspaces
    except AttributeError:
        _kept.workspaces = {}
        return _kept.workspaces


def _own_workspace(nbytes: int, device: int, stream: int) -> torch.Tensor:
    """The workspace of an attention call that was given none: one per device, stream and thread, so that
    calls that overlap share none, kept until the thread ends; while the stream is captured a new one,
    owned by the graph.  Of that one only the header, with the error word, is zeroed on every replay: the
    plan writes the rest before it is read."""
    if torch.cuda.is_current_stream_capturing():
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        ws[:256].zero_()
        return ws
    kept = _own_workspaces()
    ws = kept.get((device, stream))
    if ws is None or ws.numel() < nbytes:
        ws = kept[device, stream] = torch.zeros(nbytes, dtype=torch.uint8, device=device)
    return ws


def _kv_code(dtype) -> int:
    if dtype == torch.bfloat16:
        return BF16
    if dtype == torch.float8_e4m3fn:
        return FP8_E4M3
    if dtype == torch.int8:
        return INT8
    if dtype == torch.uint8:  # int4 values packed two a byte (element 2i in the low nibble of byte i)
        return INT4
    raise ValueError(f"unsupported KV dtype {dtype}")


def kv_head_dim(kv_pages) -> int:
    """Head dim of a cache tensor: its last dim, twice that for a packed int4 (uint8) cache."""
    return kv_pages.shape[-1] * (2 if kv_pages.dtype == torch.uint8 else 1)


def make_rpa_params(q, kv_pages, page_indices, *, sm_scale=1.0, sliding_window=None, soft_cap=None,
                    mask_value=None, k_scale=None, v_scale=None, batch_kind=BATCH_MIXED) -> rpa_params:
    P, ps, C, _ = kv_pages.shape
    D = kv_head_dim(kv_pages)
    max_num_seqs, pps = page_indices.shape
    return rpa_params(
        struct_size=ctypes.sizeof(rpa_params), version=ABI_VERSION, max_num_tokens=q.shape[0],
        num_q_heads=q.shape[1], num_combined_kv_heads=C, head_dim=D, total_num_pages=P, page_size=ps,
        max_num_seqs=max_num_seqs, pages_per_seq=pps, q_dtype=BF16, kv_dtype=_kv_code(kv_pages.dtype),
        sm_scale=float(sm_scale), sliding_window=int(_opt(sliding_window, 0)), soft_cap=float(_opt(soft_cap)),
        mask_value=math.nan if mask_value is None else float(mask_value), k_scale=float(_opt(k_scale)),
        v_scale=float(_opt(v_scale)), batch_kind=int(batch_kind))


def rpa_workspace_size(params: rpa_params) -> int:
    lib = load_library()
    n = ctypes.c_size_t(0)
    _check(lib.rpa_workspace_size(ctypes.byref(params), ctypes.byref(n)))
    return n.value


def rpa_forward(q, kv_pages, kv_lens, page_indices, cu_q_lens, num_seqs, *, sm_scale=1.0, sliding_window=None,
                soft_cap=None, mask_value=None, k_scale=None, v_scale=None, out=None, workspace=None,
                batch_kind=BATCH_MIXED):
    """Ragged paged attention; returns ``out`` [max_num_tokens, Hq, D] bf16.  ``batch_kind``
    (BATCH_DECODE_ONLY / BATCH_PREFILL_ONLY) lets the library skip the other class's launches."""
    lib = load_library()
    _dev(q, "q", torch.bfloat16)
    _dev(kv_pages, "kv_pages")
    for n, t in (("kv_lens", kv_lens), ("page_indices", page_indices), ("cu_q_lens", cu_q_lens),
                 ("num_seqs", num_seqs)):
        _dev(t, n, torch.int32)
    prm = make_rpa_params(q, kv_pages, page_indices, sm_scale=sm_scale, sliding_window=sliding_window,
                          soft_cap=soft_cap, mask_value=mask_value, k_scale=k_scale, v_scale=v_scale,
                          batch_kind=batch_kind)
    if kv_lens.numel() != prm.max_num_seqs or cu_q_lens.numel() != prm.max_num_seqs + 1 or num_seqs.numel() != 1:
        raise ValueError("kv_lens must be [max_num_seqs], cu_q_lens [max_num_seqs + 1], num_seqs [1]")
    if kv_head_dim(kv_pages) != q.shape[-1]:
        raise ValueError("q and kv_pages head_dim differ")
    if out is None:
        out = torch.empty_like(q)
    elif tuple(out.shape) != tuple(q.shape):
        raise ValueError(f"out must have q's shape {tuple(q.shape)}, got {tuple(out.shape)}")
    _dev(out, "out", torch.bfloat16)
    if workspace is None:
        workspace = Workspace.get(rpa_workspace_size(prm), q.device, "rpa")
    _check(lib.rpa_forward(ctypes.byref(prm), _ptr(q), _ptr(kv_pages), _ptr(kv_lens), _ptr(page_indices),
                           _ptr(cu_q_lens), _ptr(num_seqs), _ptr(out), _ptr(workspace), workspace.numel(),
                           _stream()))
    return out


def _header_noalloc_bytes() -> int:
    """RPA_NOALLOC_SCRATCH_BYTES as ``include/rpa.h`` defines it (the one definition of the
    size; the binding reads it instead of restating it)."""
    path = os.path.join(os.path.dirname(_HERE), "include", "rpa.h")
    with open(path) as f:
        m = re.search(r"#define\s+RPA_NOALLOC_SCRATCH_BYTES\s+\((\d+)u\s*<<\s*(\d+)\)", f.read())
    if m is None:
        raise RuntimeError(f"RPA_NOALLOC_SCRATCH_BYTES not found in {path}")
    return int(m.group(1)) << int(m.group(2))


NOALLOC_SCRATCH_BYTES = _header_noalloc_bytes()


def rpa_forward_noalloc(q, kv_pages, kv_lens, page_indices, cu_q_lens, num_seqs, *, out, sm_scale=1.0,
                        sliding_window=None, soft_cap=None, mask_value=None, k_scale=None, v_scale=None):
    """rpa_forward through the entry point that allocates nothing.

    For callers that cannot allocate device memory (their host application's memory
    manager owns the GPU, or allocation is not allowed once serving has started): the
    library uses its own fixed scratch array instead of a workspace, so ``out`` must be
    given.  Overlapping calls race on that array; problems needing more than
    ``NOALLOC_SCRATCH_BYTES`` of scratch raise ``RpaError`` (RPA_ERR_WORKSPACE).
    """
    # shapes first: the C call sees only pointers, so a q narrower than the cache or an
    # out smaller than q would be read or written past its end
    if kv_head_dim(kv_pages) != q.shape[-1]:
        raise ValueError("q and kv_pages head_dim differ")
    if tuple(out.shape) != tuple(q.shape):
        raise ValueError(f"out must have q's shape {tuple(q.shape)}, got {tuple(out.shape)}")
    lib = load_library()
    _dev(q, "q", torch.bfloat16)
    _dev(kv_pages, "kv_pages")
    _dev(out, "out", torch.bfloat16)
    for n, t in (("kv_lens", kv_lens), ("page_indices", page_indices), ("cu_q_lens", cu_q_lens),
                 ("num_seqs", num_seqs)):
        _dev(t, n, torch.int32)
    prm = make_rpa_params(q, kv_pages, page_indices, sm_scale=sm_scale, sliding_window=sliding_window,
                          soft_cap=soft_cap, mask_value=mask_value, k_scale=k_scale, v_scale=v_scale)
    if kv_lens.numel() != prm.max_num_seqs or cu_q_lens.numel() != prm.max_num_seqs + 1 or num_seqs.numel() != 1:
        raise ValueError("kv_lens must be [max_num_seqs], cu_q_lens [max_num_seqs + 1], num_seqs [1]")
    _check(lib.rpa_forward_noalloc(ctypes.byref(prm), _ptr(q), _ptr(kv_pages), _ptr(kv_lens), _ptr(page_indices),
                                   _ptr(cu_q_lens), _ptr(num_seqs), _ptr(out), _stream()))
    return out


def rpa_update_kv_cache(new_k, new_v, kv_pages, kv_lens, page_indices, cu_q_lens, num_seqs, *, workspace=None):
    """Scatter new K/V [max_num_tokens, Hkv, D] into ``kv_pages`` in place; returns ``kv_pages``."""
    lib = load_library()
    _dev(kv_pages, "kv_pages")
    _dev(new_k, "new_k", kv_pages.dtype)
    _dev(new_v, "new_v", kv_pages.dtype)
    for n, t in (("kv_lens", kv_lens), ("page_indices", page_indices), ("cu_q_lens", cu_q_lens),
                 ("num_seqs", num_seqs)):
        _dev(t, n, torch.int32)
    if new_k.shape != new_v.shape or new_k.shape[1] * 2 != kv_pages.shape[2] or new_k.shape[2] != kv_pages.shape[3]:
        raise ValueError("new_k/new_v must be [max_num_tokens, num_kv_heads, head_dim]")
    fake_q = torch.empty((new_k.shape[0], new_k.shape[1]), device="meta")
    prm = make_rpa_params(fake_q, kv_pages, page_indices)
    if workspace is None:
        workspace = Workspace.get(256, kv_pages.device, "update")
    _check(lib.rpa_update_kv_cache(ctypes.byref(prm), _ptr(new_k), _ptr(new_v), _ptr(kv_pages), _ptr(kv_lens),
                                   _ptr(page_indices), _ptr(cu_q_lens), _ptr(num_seqs), _ptr(workspace),
                                   workspace.numel(), _stream()))
    return kv_pages


def rpa_forward_update(q, new_k, new_v, kv_pages, kv_lens, page_indices, cu_q_lens, num_seqs, *, sm_scale=1.0,
                       sliding_window=None, soft_cap=None, mask_value=None, k_scale=None, v_scale=None, out=None,
                       workspace=None, batch_kind=BATCH_MIXED):
    """rpa_update_kv_cache then rpa_forward in one call (the cache write shares the plan's
    launch); writes ``kv_pages`` in place and returns ``out``."""
    lib = load_library()
    _dev(q, "q", torch.bfloat16)
    _dev(kv_pages, "kv_pages")
    _dev(new_k, "new_k", kv_pages.dtype)
    _dev(new_v, "new_v", kv_pages.dtype)
    for n, t in (("kv_lens", kv_lens), ("page_indices", page_indices), ("cu_q_lens", cu_q_lens),
                 ("num_seqs", num_seqs)):
        _dev(t, n, torch.int32)
    prm = make_rpa_params(q, kv_pages, page_indices, sm_scale=sm_scale, sliding_window=sliding_window,
                          soft_cap=soft_cap, mask_value=mask_value, k_scale=k_scale, v_scale=v_scale,
                          batch_kind=batch_kind)
    if kv_lens.numel() != prm.max_num_seqs or cu_q_lens.numel() != prm.max_num_seqs + 1 or num_seqs.numel() != 1:
        raise ValueError("kv_lens must be [max_num_seqs], cu_q_lens [max_num_seqs + 1], num_seqs [1]")
    if kv_head_dim(kv_pages) != q.shape[-1]:
        raise ValueError("q and kv_pages head_dim differ")
    if (new_k.shape != new_v.shape or new_k.shape[0] != q.shape[0] or new_k.shape[1] * 2 != kv_pages.shape[2]
            or new_k.shape[2] != kv_pages.shape[3]):
        raise ValueError("new_k/new_v must be [max_num_tokens, num_kv_heads, head_dim]")
    if out is None:
        out = torch.empty_like(q)
    elif tuple(out.shape) != tuple(q.shape):
        raise ValueError(f"out must have q's shape {tuple(q.shape)}, got {tuple(out.shape)}")
    _dev(out, "out", torch.bfloat16)
    if workspace is None:
        workspace = Workspace.get(rpa_workspace_size(prm), q.device, "rpa")
    _check(lib.rpa_forward_update(ctypes.byref(prm), _ptr(q), _ptr(new_k), _ptr(new_v), _ptr(kv_pages),
                                  _ptr(kv_lens), _ptr(page_indices), _ptr(cu_q_lens), _ptr(num_seqs), _ptr(out),
                                  _ptr(workspace), workspace.numel(), _stream()))
    return out


def make_rope_table(rotary_dim, *, base=10000.0, interleaved=False, scaling=None) -> rope_table:
    """The table the rotating calls take; made once from the model's configuration.

    ``scaling`` names a change of the frequencies and its numbers, as ``include/rpa.h`` defines them:
    ``{"type": "linear" | "ntk", "factor": ...}``, ``{"type": "llama3", "factor", "low_freq_factor",
    "high_freq_factor", "original_max_position"}`` or ``{"type": "yarn", "factor", "beta_fast" (32),
    "beta_slow" (1), "original_max_position"}``; each may carry ``"attention_factor"``, the factor on
    every turned element (YaRN's default is 0.1 ln(factor) + 1)."""
    more = dict(scaling or {"type": "none"})
    kind = more.pop("type", None)
    if kind not in ROPE_SCALINGS:
        raise ValueError(f"scaling type {kind!r} is none of {sorted(ROPE_SCALINGS)}")
    takes = {"none": (), "linear": ("factor",), "ntk": ("factor",),
             "llama3": ("factor", "low_freq_factor", "high_freq_factor", "original_max_position"),
             "yarn": ("factor", "beta_fast", "beta_slow", "original_max_position")}[kind]
    if kind == "yarn":
        more = {"beta_fast": 32.0, "beta_slow": 1.0, **more}
    if set(more) - {"attention_factor"} != set(takes):
        raise ValueError(f"{kind} scaling takes {', '.join(takes) or 'nothing'} (and attention_factor), got {sorted(more)}")
    p = rope_params(struct_size=ctypes.sizeof(rope_params), version=ABI_VERSION, rotary_dim=int(rotary_dim),
                    pairing=ROPE_INTERLEAVED if interleaved else ROPE_HALF, scaling=ROPE_SCALINGS[kind], base=float(base))
    for name, value in more.items():
        setattr(p, name, int(value) if name == "original_max_position" else float(value))
    t = rope_table()
    _check(load_library().rope_table_init(ctypes.byref(p), ctypes.byref(t)))
    return t


def _rows(t, name: str, device: int, heads: int = 0, dim: int = 0):
    """(token stride, head stride) of bf16 rows [tokens, heads, head_dim] on ``device``; any strides with
    adjacent elements and 16-byte aligned rows.  ``heads`` and ``dim``, where given, must match."""
    try:
        n, h, d = t.shape
        token, head, element = t.stride()
        good = t.dtype is _BF16 and t.get_device() == device
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        raise ValueError(f"{name} must be a bfloat16 CUDA tensor [tokens, heads, head_dim] on device {device}")
    if (heads and h != heads) or (dim and d != dim):
        raise ValueError(f"{name} must have {heads or h} heads of {dim or d}, got {tuple(t.shape)}")
    if h <= 1:  # the stride of a dimension of one entry says nothing
        head = d
    if n <= 1:
        token = h * head
    if element != 1 or head % 8 or token % 8 or head <= 0 or token <= 0:
        raise ValueError(f"{name} must have adjacent elements and token and head strides that are positive multiples "
                         f"of 8, got strides {t.stride()}")
    return token, head


def _on(device: int, t, name: str, dtype, n: int = -1):
    """Checks a contiguous tensor of ``dtype`` on ``device`` (of ``n`` elements, where given)."""
    try:
        good = t.dtype is dtype and t.get_device() == device and t.is_contiguous()
    except AttributeError:
        good = False
    if not good:
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor on device {device}")
    if n >= 0 and t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, got shape {tuple(t.shape)}")


def _cuda_index(t, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _is_table(table):
    if not isinstance(table, rope_table):
        raise ValueError("table must come from make_rope_table")


def rope_apply(q, k, positions, table, *, inverse=False, q_out=None, k_out=None):
    """Turns q [T, Hq, D] and k [T, Hk, D] (or None) to ``positions`` [T] int32; returns ``(q_out, k_out)``.

    q and k are bf16 with any token and head strides; ``q_out=q`` and ``k_out=k`` work in place.
    ``inverse`` turns back by the same angles (the map of an output's gradient to the input's).  Autograd does
    not see the call: outputs carry no history, and a turn in place leaves the tensor's version as it was; a
    training program calls it and its inverse from an ``autograd.Function`` of its own."""
    lib = _lib or load_library()
    _is_table(table)
    dev = _cuda_index(q, "q")
    if dev != _current():
        with torch.cuda.device(dev):
            return rope_apply(q, k, positions, table, inverse=inverse, q_out=q_out, k_out=k_out)
    q_token, q_head = _rows(q, "q", dev)
    T, hq, d = q.shape
    _on(dev, positions, "positions", _I32, T)
    if q_out is None:
        q_out = torch.empty((T, hq, d), dtype=torch.bfloat16, device=q.device)
    qo_token, qo_head = (q_token, q_head) if q_out is q else _rows(q_out, "q_out", dev)
    if q_out.shape != q.shape:
        raise ValueError(f"q_out must have q's shape {tuple(q.shape)}, got {tuple(q_out.shape)}")
    hk = k_token = k_head = ko_token = ko_head = 0
    if k is not None:
        k_token, k_head = _rows(k, "k", dev, 0, d)
        hk = k.shape[1]
        if k_out is None:
            k_out = torch.empty((T, hk, d), dtype=torch.bfloat16, device=q.device)
        ko_token, ko_head = (k_token, k_head) if k_out is k else _rows(k_out, "k_out", dev)
        if k.shape[0] != T or k_out.shape != k.shape:
            raise ValueError(f"k and k_out must be [{T}, heads, {d}], got {tuple(k.shape)} and {tuple(k_out.shape)}")
    elif k_out is not None:
        raise ValueError("k_out goes with k")
    if T == 0:
        return q_out, k_out
    prm = rope_apply_params(_APPLY_SIZE, ABI_VERSION, T, hq, hk, d, 1 if inverse else 0, 0, q_token, q_head, k_token, k_head,
                            qo_token, qo_head, ko_token, ko_head)
    rc = lib.rope_apply(ctypes.byref(prm), ctypes.byref(table), q.data_ptr(), k.data_ptr() if hk else None,
                        positions.data_ptr(), q_out.data_ptr(), k_out.data_ptr() if hk else None, _raw_stream(dev))
    if rc:
        _check(rc)
    return q_out, k_out


def _batch_params(dev, tokens, hq, d, kv_pages, kv_lens, page_indices, cu_q_lens, num_seqs, sm_scale=1.0, sliding_window=None,
                  soft_cap=None, mask_value=None, k_scale=None, v_scale=None, batch_kind=BATCH_MIXED) -> rpa_params:
    """rpa_params of a batch of ``tokens`` queries of ``hq`` heads, its cache and metadata checked."""
    if not isinstance(kv_pages, torch.Tensor) or kv_pages.get_device() != dev or kv_pages.dim() != 4:
        raise ValueError(f"kv_pages must be [pages, page_size, heads, head_dim] on device {dev}")
    if not kv_pages.is_contiguous():
        raise ValueError("kv_pages must be contiguous")
    code = _kv_code(kv_pages.dtype)
    pages, ps, combined, width = kv_pages.shape
    if (width * 2 if code == INT4 else width) != d:
        raise ValueError(f"kv_pages hold heads of {kv_head_dim(kv_pages)}, the rows {d}")
    _on(dev, page_indices, "page_indices", _I32)
    if page_indices.dim() != 2:
        raise ValueError("page_indices must be [max_num_seqs, pages_per_seq]")
    seqs, pps = page_indices.shape
    _on(dev, kv_lens, "kv_lens", _I32, seqs)
    _on(dev, cu_q_lens, "cu_q_lens", _I32, seqs + 1)
    _on(dev, num_seqs, "num_seqs", _I32, 1)
    return rpa_params(_PARAMS_SIZE, ABI_VERSION, tokens, hq, combined, d, pages, ps, seqs, pps, BF16, code, sm_scale,
                      sliding_window or 0, soft_cap or 0.0, math.nan if mask_value is None else mask_value, k_scale or 0.0,
                      v_scale or 0.0, batch_kind)


_PARAMS_SIZE, _APPLY_SIZE, _STRIDES_SIZE = (ctypes.sizeof(x) for x in (rpa_params, rope_apply_params, rope_strides))


def _rope_update_args(dev, q, new_k, new_v, kv_pages, kv_lens, page_indices, cu_q_lens, num_seqs, table, positions, q_out,
                      **opts):
    """The checks the appending calls share; (rpa_params, rope_strides, q_out)."""
    _is_table(table)
    k_token, k_head = _rows(new_k, "new_k", dev)
    T, hkv, d = new_k.shape
    v_token, v_head = _rows(new_v, "new_v", dev, hkv, d)
    if new_v.shape[0] != T:
        raise ValueError("new_k and new_v must have the same number of tokens")
    q_token = q_head = 0
    if q is not None:
        q_token, q_head = _rows(q, "q", dev, 0, d)
        if q.shape[0] != T:
            raise ValueError("q must have new_k's number of tokens")
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        _on(dev, q_out, "q_out", torch.bfloat16)
        if q_out.shape != q.shape:
            raise ValueError(f"q_out must have q's shape {tuple(q.shape)}, got {tuple(q_out.shape)}")
    elif q_out is not None:
        raise ValueError("q_out goes with q")
    if positions is not None:
        _on(dev, positions, "positions", _I32, T)
    prm = _batch_params(dev, T, hkv if q is None else q.shape[1], d, kv_pages, kv_lens, page_indices, cu_q_lens, num_seqs, **opts)
    if prm.num_combined_kv_heads != 2 * hkv:
        raise ValueError(f"kv_pages have {prm.num_combined_kv_heads} combined heads, new_k and new_v {hkv} each")
    return prm, rope_strides(_STRIDES_SIZE, ABI_VERSION, q_token, q_head, k_token, k_head, v_token, v_head), q_out


def rpa_rope_update_kv_cache(q, new_k, new_v, kv_pages, kv_lens, page_indices, cu_q_lens, num_seqs, table, *,
                             positions=None, k_scale=None, v_scale=None, q_out=None, workspace=None):
    """Turns ``new_k`` [T, Hkv, D] bf16 to its slots' positions and writes it and ``new_v`` into
    ``kv_pages`` in place, rounded to the cache's type (divided by the scales first); turns ``q``
    [T, Hq, D] (or None) beside them.  Returns ``(q_out, kv_pages)``.

    q, new_k and new_v take any token and head strides (slices of one projection's output);
    ``positions`` [T] int32 turns by other positions than the slots' own.  Bad metadata is recorded in
    ``workspace``'s error word where one is given."""
    lib = _lib or load_library()
    dev = _cuda_index(new_k, "new_k")
    if dev != _current():
        with torch.cuda.device(dev):
            return rpa_rope_update_kv_cache(q, new_k, new_v, kv_pages, kv_lens, page_indices, cu_q_lens, num_seqs, table,
                                            positions=positions, k_scale=k_scale, v_scale=v_scale, q_out=q_out,
                                            workspace=workspace)
    prm, st, q_out = _rope_update_args(dev, q, new_k, new_v, kv_pages, kv_lens, page_indices, cu_q_lens, num_seqs, table,
                                       positions, q_out, k_scale=k_scale, v_scale=v_scale)
    if workspace is not None:
        _on(dev, workspace, "workspace", torch.uint8)
    if prm.max_num_tokens == 0:
        return q_out, kv_pages
    rc = lib.rpa_rope_update_kv_cache(
        ctypes.byref(prm), ctypes.byref(table), ctypes.byref(st), None if q is None else q.data_ptr(), new_k.data_ptr(),
        new_v.data_ptr(), kv_pages.data_ptr(), kv_lens.data_ptr(), page_indices.data_ptr(), cu_q_lens.data_ptr(),
        num_seqs.data_ptr(), None if positions is None else positions.data_ptr(), None if q is None else q_out.data_ptr(),
        None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel(), _raw_stream(dev))
    if rc:
        _check(rc)
    return q_out, kv_pages


def _attention_buffers(dev, size, prm, q, out, workspace):
    """(out, workspace, stream) of an attention call, made where none are given; size: its workspace query."""
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    _on(dev, out, "out", torch.bfloat16)
    if out.shape != q.shape:
        raise ValueError(f"out must have q's shape {tuple(q.shape)}, got {tuple(out.shape)}")
    stream = _raw_stream(dev)
    if workspace is not None:
        _on(dev, workspace, "workspace", torch.uint8)
    elif prm.max_num_tokens:
        n = ctypes.c_size_t(0)
        _check(size(ctypes.byref(prm), ctypes.byref(n)))
        workspace = _own_workspace(n.value, dev, stream)
    return out, workspace, stream


def rpa_rope_forward_update(q, new_k, new_v, kv_pages, kv_lens, page_indices, cu_q_lens, num_seqs, table, *,
                            positions=None, sm_scale=1.0, sliding_window=None, soft_cap=None, mask_value=None,
                            k_scale=None, v_scale=None, q_rot=None, out=None, workspace=None, batch_kind=BATCH_MIXED):
    """rpa_rope_update_kv_cache, then rpa_forward of the turned queries (kept in ``q_rot``), in one call;
    writes ``kv_pages`` in place and returns ``out`` [T, Hq, D]."""
    lib = _lib or load_library()
    dev = _cuda_index(q, "q")
    if dev != _current():
        with torch.cuda.device(dev):
            return rpa_rope_forward_update(q, new_k, new_v, kv_pages, kv_lens, page_indices, cu_q_lens, num_seqs, table,
                                           positions=positions, sm_scale=sm_scale, sliding_window=sliding_window,
                                           soft_cap=soft_cap, mask_value=mask_value, k_scale=k_scale, v_scale=v_scale,
                                           q_rot=q_rot, out=out, workspace=workspace, batch_kind=batch_kind)
    prm, st, q_rot = _rope_update_args(dev, q, new_k, new_v, kv_pages, kv_lens, page_indices, cu_q_lens, num_seqs, table,
                                       positions, q_rot, sm_scale=sm_scale, sliding_window=sliding_window,
                                       soft_cap=soft_cap, mask_value=mask_value, k_scale=k_scale, v_scale=v_scale,
                                       batch_kind=batch_kind)
    out, workspace, stream = _attention_buffers(dev, lib.rpa_workspace_size, prm, q, out, workspace)
    if prm.max_num_tokens == 0:
        return out
    rc = lib.rpa_rope_forward_update(
        ctypes.byref(prm), ctypes.byref(table), ctypes.byref(st), q.data_ptr(), new_k.data_ptr(), new_v.data_ptr(),
        kv_pages.data_ptr(), kv_lens.data_ptr(), page_indices.data_ptr(), cu_q_lens.data_ptr(), num_seqs.data_ptr(),
        None if positions is None else positions.data_ptr(), q_rot.data_ptr(), out.data_ptr(), workspace.data_ptr(),
        workspace.numel(), stream)
    if rc:
        _check(rc)
    return out


def rpa_cross_workspace_size(params: rpa_params) -> int:
    lib = load_library()
    n = ctypes.c_size_t(0)
    _check(lib.rpa_cross_workspace_size(ctypes.byref(params), ctypes.byref(n)))
    return n.value


def rpa_cross_forward(q, kv_pages, kv_lens, page_indices, cu_q_lens, num_seqs, *, sm_scale=1.0, soft_cap=None,
                      k_scale=None, v_scale=None, out=None, workspace=None, batch_kind=BATCH_MIXED):
    """Attention of every query to all ``kv_lens`` keys of its sequence (a decoder's tokens to its
    encoder's states); returns ``out`` [max_num_tokens, Hq, D] bf16.  A sequence without keys gets zeros."""
    lib = _lib or load_library()
    dev = _cuda_index(q, "q")
    if dev != _current():
        with torch.cuda.device(dev):
            return rpa_cross_forward(q, kv_pages, kv_lens, page_indices, cu_q_lens, num_seqs, sm_scale=sm_scale,
                                     soft_cap=soft_cap, k_scale=k_scale, v_scale=v_scale, out=out, workspace=workspace,
                                     batch_kind=batch_kind)
    _on(dev, q, "q", torch.bfloat16)
    if q.dim() != 3:
        raise ValueError(f"q must be [tokens, heads, head_dim], got {tuple(q.shape)}")
    T, hq, d = q.shape
    prm = _batch_params(dev, T, hq, d, kv_pages, kv_lens, page_indices, cu_q_lens, num_seqs, sm_scale, None, soft_cap, None,
                        k_scale, v_scale, batch_kind)
    out, workspace, stream = _attention_buffers(dev, lib.rpa_cross_workspace_size, prm, q, out, workspace)
    if T == 0:
        return out
    rc = lib.rpa_cross_forward(ctypes.byref(prm), q.data_ptr(), kv_pages.data_ptr(), kv_lens.data_ptr(), page_indices.data_ptr(),
                               cu_q_lens.data_ptr(), num_seqs.data_ptr(), out.data_ptr(), workspace.data_ptr(),
                               workspace.numel(), stream)
    if rc:
        _check(rc)
    return out


def make_mla_params(ql_nope, q_pe, cache_kv_c, cache_k_pe, kv_lens, page_indices, *, sm_scale=1.0,
                    sliding_window=None, soft_cap=None, mask_value=None, q_scale=None) -> mla_params:
    P, ps_pk, pk, lkv_pad = cache_kv_c.shape
    max_num_seqs = kv_lens.numel()
    fp8 = ql_nope.dtype == torch.float8_e4m3fn
    return mla_params(
        struct_size=ctypes.sizeof(mla_params), version=ABI_VERSION, max_num_tokens=ql_nope.shape[0],
        num_q_heads=ql_nope.shape[1], lkv_dim=ql_nope.shape[2], r_dim=q_pe.shape[2], lkv_dim_pad=lkv_pad,
        r_dim_pad=cache_k_pe.shape[-1], total_num_pages=P, page_size=ps_pk * pk, kv_packing=pk,
        max_num_seqs=max_num_seqs, pages_per_seq=page_indices.numel() // max_num_seqs, sm_scale=float(sm_scale),
        sliding_window=int(_opt(sliding_window, 0)), soft_cap=float(_opt(soft_cap)),
        mask_value=math.nan if mask_value is None else float(mask_value),
        q_dtype=FP8_E4M3 if fp8 else BF16, q_scale=float(_opt(q_scale)) if fp8 else 0.0)


def mla_workspace_size(params: mla_params) -> int:
    lib = load_library()
    n = ctypes.c_size_t(0)
    _check(lib.mla_workspace_size(ctypes.byref(params), ctypes.byref(n)))
    return n.value


def _check_mla(ql_nope, q_pe, new_kv_c, new_k_pe, cache_kv_c, cache_k_pe, kv_lens, page_indices, cu_q_lens,
               distribution):
    qdt = torch.float8_e4m3fn if ql_nope.dtype == torch.float8_e4m3fn else torch.bfloat16
    for n, t in (("ql_nope", ql_nope), ("q_pe", q_pe)):
        _dev(t, n, qdt)
    for n, t in (("new_kv_c", new_kv_c), ("new_k_pe", new_k_pe), ("cache_kv_c", cache_kv_c),
                 ("cache_k_pe", cache_k_pe)):
        _dev(t, n, torch.bfloat16)
    for n, t in (("kv_lens", kv_lens), ("page_indices", page_indices), ("cu_q_lens", cu_q_lens),
                 ("distribution", distribution)):
        _dev(t, n, torch.int32)
    if cu_q_lens.numel() != kv_lens.numel() + 1 or distribution.numel() != 3:
        raise ValueError("cu_q_lens must be [max_num_seqs + 1] and distribution [3]")
    if page_indices.numel() % kv_lens.numel():
        raise ValueError("page_indices must hold max_num_seqs * pages_per_seq entries")


def mla_update_kv_cache(new_kv_c, new_k_pe, cache_kv_c, cache_k_pe, kv_lens, page_indices, cu_q_lens,
                        distribution, *, workspace=None):
    """MLA cache scatter, in place; returns ``(cache_kv_c, cache_k_pe)``."""
    lib = load_library()
    T = new_kv_c.shape[0]
    fake_ql = torch.empty((T, 1, new_kv_c.shape[1]), device="meta")
    fake_qr = torch.empty((T, 1, new_k_pe.shape[1]), device="meta")
    _check_mla(new_kv_c.unsqueeze(1), new_k_pe.unsqueeze(1), new_kv_c, new_k_pe, cache_kv_c, cache_k_pe, kv_lens,
               page_indices, cu_q_lens, distribution)
    prm = make_mla_params(fake_ql, fake_qr, cache_kv_c, cache_k_pe, kv_lens, page_indices)
    if workspace is None:
        workspace = Workspace.get(256, cache_kv_c.device, "update")
    _check(lib.mla_update_kv_cache(ctypes.byref(prm), _ptr(new_kv_c), _ptr(new_k_pe), _ptr(cache_kv_c),
                                   _ptr(cache_k_pe), _ptr(kv_lens), _ptr(page_indices), _ptr(cu_q_lens),
                                   _ptr(distribution), _ptr(workspace), workspace.numel(), _stream()))
    return cache_kv_c, cache_k_pe


def mla_rpa_forward(ql_nope, q_pe, new_kv_c, new_k_pe, cache_kv_c, cache_k_pe, kv_lens, page_indices, cu_q_lens,
                    distribution, *, sm_scale=1.0, sliding_window=None, soft_cap=None, mask_value=None, q_scale=None,
                    out=None, workspace=None):
    """MLA update_kv_cache + attention; returns ``out`` [max_num_tokens, H, lkv] bf16 (caches updated in place).

    ``ql_nope`` and ``q_pe`` are bf16, or both float8_e4m3fn with ``q_scale`` multiplying the
    scores after ``sm_scale``."""
    lib = load_library()
    _check_mla(ql_nope, q_pe, new_kv_c, new_k_pe, cache_kv_c, cache_k_pe, kv_lens, page_indices, cu_q_lens,
               distribution)
    if q_scale is not None and ql_nope.dtype != torch.float8_e4m3fn:
        raise ValueError("q_scale applies to float8_e4m3fn queries only")
    prm = make_mla_params(ql_nope, q_pe, cache_kv_c, cache_k_pe, kv_lens, page_indices, sm_scale=sm_scale,
                          sliding_window=sliding_window, soft_cap=soft_cap, mask_value=mask_value, q_scale=q_scale)
    if out is None:
        out = torch.empty(ql_nope.shape, dtype=torch.bfloat16, device=ql_nope.device)
    _dev(out, "out", torch.bfloat16)
    if workspace is None:
        workspace = Workspace.get(mla_workspace_size(prm), ql_nope.device, "mla")
    _check(lib.mla_rpa_forward(ctypes.byref(prm), _ptr(ql_nope), _ptr(q_pe), _ptr(new_kv_c), _ptr(new_k_pe),
                               _ptr(cache_kv_c), _ptr(cache_k_pe), _ptr(kv_lens), _ptr(page_indices),
                               _ptr(cu_q_lens), _ptr(distribution), _ptr(out), _ptr(workspace), workspace.numel(),
                               _stream()))
    return out


def make_sparse_params(q, cache, indices, page_table, *, read_block, page_size, seq_len, sm_scale,
                       dv=512) -> sparse_params:
    B, S, H, Dk = q.shape
    row_stride = cache.shape[-1]
    P = cache.numel() // (page_size * row_stride)
    return sparse_params(
        struct_size=ctypes.sizeof(sparse_params), version=ABI_VERSION, batch=B, num_queries=S, num_heads=H, dk=Dk,
        dv=dv, row_stride=row_stride, topk=indices.shape[-1], read_block=read_block, page_size=page_size,
        max_pages=page_table.shape[-1], total_num_pages=P, seq_len=seq_len, sm_scale=float(sm_scale))


def sparse_mla_workspace_size(params: sparse_params) -> int:
    lib = load_library()
    n = ctypes.c_size_t(0)
    _check(lib.sparse_mla_workspace_size(ctypes.byref(params), ctypes.byref(n)))
    return n.value


def sparse_mla_forward(q, cache, indices, positions, page_table, *, read_block, page_size, seq_len, sm_scale,
                       dv=512, out=None, workspace=None):
    """DSA sparse MLA; returns ``out`` [B, S, H, dv] float32."""
    lib = load_library()
    _dev(q, "q", torch.bfloat16)
    _dev(cache, "cache", torch.bfloat16)
    for n, t in (("indices", indices), ("positions", positions), ("page_table", page_table)):
        _dev(t, n, torch.int32)
    B, S, H, _ = q.shape
    if indices.shape[:2] != (B, S) or positions.shape != (B, S) or page_table.shape[0] != B:
        raise ValueError("indices [B, S, K], positions [B, S] and page_table [B, max_pages] must match q")
    if sm_scale is None:
        raise ValueError("sm_scale is required")
    prm = make_sparse_params(q, cache, indices, page_table, read_block=read_block, page_size=page_size,
                             seq_len=seq_len, sm_scale=sm_scale, dv=dv)
    if out is None:
        out = torch.empty((B, S, H, dv), dtype=torch.float32, device=q.device)
    _dev(out, "out", torch.float32)
    if workspace is None:
        workspace = Workspace.get(sparse_mla_workspace_size(prm), q.device, "sparse")
    _check(lib.sparse_mla_forward(ctypes.byref(prm), _ptr(q), _ptr(cache), _ptr(indices), _ptr(positions),
                                  _ptr(page_table), _ptr(out), _ptr(workspace), workspace.numel(), _stream()))
    return out


def make_sparse_ragged_params(ql, qpe, cache, topk, seq_lens, page_indices, *, read_block, page_size,
                              sm_scale) -> sparse_ragged_params:
    T, H, dv = ql.shape
    row_stride = cache.shape[-1]
    return sparse_ragged_params(
        struct_size=ctypes.sizeof(sparse_ragged_params), version=ABI_VERSION, num_tokens=T, num_seqs=seq_lens.numel(),
        num_heads=H, dv=dv, rope=qpe.shape[-1], row_stride=row_stride, topk=topk.shape[-1], read_block=read_block,
        page_size=page_size, num_page_ids=page_indices.numel(),
        total_num_pages=cache.numel() // (page_size * row_stride), sm_scale=float(sm_scale))


def sparse_mla_ragged_workspace_size(params: sparse_ragged_params) -> int:
    lib = load_library()
    n = ctypes.c_size_t(0)
    _check(lib.sparse_mla_ragged_workspace_size(ctypes.byref(params), ctypes.byref(n)))
    return n.value


def sparse_mla_write_and_attend_ragged(ql, qpe, kvc, kpe, cache, topk, positions, loc, seq_lens, cu_q_lens,
                                       cu_kv_lens, page_indices, *, read_block, page_size, sm_scale, out=None,
                                       workspace=None):
    """Packed-ragged sparse MLA with the self-write: writes ``kvc``/``kpe`` rows (may be None,
    with ``loc``) into ``cache`` in place, then attends; returns ``out`` [T, H, dv] float32."""
    lib = load_library()
    for n, t in (("ql", ql), ("qpe", qpe), ("cache", cache)):
        _dev(t, n, torch.bfloat16)
    for n, t in (("topk", topk), ("positions", positions), ("seq_lens", seq_lens), ("cu_q_lens", cu_q_lens),
                 ("cu_kv_lens", cu_kv_lens), ("page_indices", page_indices)):
        _dev(t, n, torch.int32)
    T, H, dv = ql.shape
    if qpe.shape[:2] != (T, H) or topk.shape[0] != T or positions.numel() != T:
        raise ValueError("qpe [T, H, rope], topk [T, K] and positions [T] must match ql [T, H, dv]")
    if cu_q_lens.numel() != seq_lens.numel() + 1 or cu_kv_lens.numel() != seq_lens.numel() + 1:
        raise ValueError("cu_q_lens and cu_kv_lens must have num_seqs + 1 entries")
    if (kvc is None) != (kpe is None) or (kvc is None) != (loc is None):
        raise ValueError("kvc, kpe and loc go together")
    if kvc is not None:
        _dev(kvc, "kvc", torch.bfloat16)
        _dev(kpe, "kpe", torch.bfloat16)
        _dev(loc, "loc", torch.int32)
        if kvc.shape != (T, dv) or kpe.shape != (T, qpe.shape[-1]) or loc.numel() != T:
            raise ValueError("kvc [T, dv], kpe [T, rope] and loc [T] must match ql")
    if sm_scale is None:
        raise ValueError("sm_scale is required")
    prm = make_sparse_ragged_params(ql, qpe, cache, topk, seq_lens, page_indices, read_block=read_block,
                                    page_size=page_size, sm_scale=sm_scale)
    if out is None:
        out = torch.empty((T, H, dv), dtype=torch.float32, device=ql.device)
    _dev(out, "out", torch.float32)
    if workspace is None:
        workspace = Workspace.get(sparse_mla_ragged_workspace_size(prm), ql.device, "sparse_ragged")
    _check(lib.sparse_mla_write_and_attend_ragged(
        ctypes.byref(prm), _ptr(ql), _ptr(qpe), _ptr(kvc), _ptr(kpe), _ptr(cache), _ptr(topk), _ptr(positions),
        _ptr(loc), _ptr(seq_lens), _ptr(cu_q_lens), _ptr(cu_kv_lens), _ptr(page_indices), _ptr(out),
        _ptr(workspace), workspace.numel(), _stream()))
    return out


def selftest_bounded_wait(workspace: torch.Tensor) -> None:
    """Launch the failure-path check (a bounded wait that runs out after 2 s and records
    RPA_DEV_ERR_TIMEOUT in ``workspace``'s error word)."""
    _check(load_library().rpa_selftest_bounded_wait(_ptr(workspace), workspace.numel(), _stream()))


def check_device_status(workspace: torch.Tensor | None = None) -> int:
    """Synchronise, read and clear the workspace error word; returns its bits (0 = fine).

    Without a workspace: that of this thread's ``rpa_cross_forward`` and ``rpa_rope_forward_update`` calls on
    the current stream that were given none.  (A captured call's own workspace is the graph's: give it one
    to read its word.)"""
    lib = load_library()
    if workspace is None:
        device = _current()
        workspace = _own_workspaces().get((device, _raw_stream(device)))
        if workspace is None:
            return 0
    bits = ctypes.c_uint32(0)
    rc = lib.rpa_check_device_status(_ptr(workspace), ctypes.byref(bits), _stream())
    if rc not in (0, -7):
        _check(rc)
    return bits.value


def launch_count() -> int:
    """Kernels the library has launched since it was loaded (``rpa_launch_count``)."""
    return int(load_library().rpa_launch_count())


class KernelTimer:
    """Per-kernel CUDA-event timing of the library's own launches (``rpa_profile_*``).

    ``with KernelTimer() as kt: ...`` then ``kt.result`` maps kernel name to
    ``(launches, total_ms)``.
    """

    def __enter__(self):
        lib = load_library()
        _check(lib.rpa_profile_reset())
        _check(lib.rpa_profile_enable(1))
        self.result = {}
        return self

    def __exit__(self, *exc):
        lib = load_library()
        _check(lib.rpa_profile_enable(0))
        n = ctypes.c_int(0)
        buf = (rpa_kernel_time * 64)()
        _check(lib.rpa_profile_read(buf, 64, ctypes.byref(n)))
        self.result = {buf[i].name.decode(): (int(buf[i].launches), float(buf[i].total_ms))
                       for i in range(min(n.value, 64))}
        _check(lib.rpa_profile_reset())
        return False
