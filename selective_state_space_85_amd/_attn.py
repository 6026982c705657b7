"""ctypes view of libssscan.so's linear-attention operators (the C ABI declared in include/ss_attn.h)."""
from __future__ import annotations

import ctypes

from . import _lib

# Every function the header declares.
EXPORTS = ("ss_lattn_workspace_bytes", "ss_lattn_fwd", "ss_lattn_bwd_workspace_bytes", "ss_lattn_bwd", "ss_lattn_step",
           "ss_qknorm_fwd", "ss_qknorm_bwd_workspace_bytes", "ss_qknorm_bwd", "ss_sample_workspace_bytes", "ss_sample")

_bound = None


def load() -> ctypes.CDLL:
    """The library (``_lib.load``) with this header's prototypes bound."""
    global _bound
    lib = _lib.load()
    if _bound is lib:
        return lib
    i64, vp, sz, ci, cf = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
    for name, args in (("ss_lattn_workspace_bytes", [i64] * 6 + [ci]), ("ss_lattn_bwd_workspace_bytes", [i64] * 6 + [ci]),
                       ("ss_qknorm_bwd_workspace_bytes", [i64] * 4), ("ss_sample_workspace_bytes", [i64] * 2 + [ci])):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, sz
    qkv = [vp, i64, vp, i64, vp, i64, vp, cf]                   # q, k, v with their row strides, log_decay, scale
    norm = [vp, i64, vp, i64, vp, vp, vp, vp, cf, ci]           # q, k with their row strides, weights, positions, eps
    for name, args in (("ss_lattn_fwd", qkv + [vp] * 5 + [sz] + [i64] * 6 + [ci, vp]),
                       ("ss_lattn_bwd", qkv + [vp] * 3 + [i64] + [vp] * 6 + [sz] + [i64] * 6 + [ci, vp]),
                       ("ss_lattn_step", [vp] + qkv + [vp] + [i64] * 5 + [ci, vp]),
                       ("ss_qknorm_fwd", norm + [vp] * 2 + [i64] * 5 + [ci, vp]),
                       ("ss_qknorm_bwd", norm + [vp] * 7 + [sz] + [i64] * 5 + [ci, vp]),
                       ("ss_sample", [vp, i64, vp, vp, cf, vp, ctypes.c_int32, vp, cf, vp, cf, vp, vp, sz] + [i64] * 2
                        + [ci, vp])):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, ci
    _bound = lib
    return lib
