"""GB300-native ragged paged attention (RPA), MLA latent RPA and DSA sparse MLA.

The compute path is a C-ABI shared library of hand-written sm_103a CUDA
kernels (``csrc/``, declared in ``include/rpa.h``).  ``api`` is the thin Python
binding over it: it marshals torch tensors into pointers and sizes and calls the
library; it performs none of the attention arithmetic itself.
"""
from .api import (RpaError, Workspace, check_device_status, load_library, make_rope_table,  # noqa: F401
                  mla_rpa_forward, mla_update_kv_cache, rope_apply, rpa_cross_forward, rpa_forward,
                  rpa_rope_forward_update, rpa_rope_update_kv_cache, rpa_update_kv_cache, sparse_mla_forward)
