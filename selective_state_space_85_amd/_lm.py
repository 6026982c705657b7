"""ctypes view of libssscan.so's language-model operators (the C ABI declared in include/ss_lm.h)."""
from __future__ import annotations

import ctypes

from . import _lib

# Every function the header declares.
EXPORTS = ("ss_glr_ckpt_bytes", "ss_glr_workspace_bytes", "ss_glr_fwd", "ss_glr_bwd_workspace_bytes", "ss_glr_bwd",
           "ss_glr_step", "ss_glu_workspace_bytes", "ss_glu_fwd", "ss_glu_bwd_workspace_bytes", "ss_glu_bwd",
           "ss_xent_workspace_bytes", "ss_xent_fwd", "ss_xent_bwd_workspace_bytes", "ss_xent_bwd")
SS_ACT_SILU, SS_ACT_GELU = 0, 1  # ss_activation

_bound = None


def load() -> ctypes.CDLL:
    """The library (``_lib.load``) with this header's prototypes bound."""
    global _bound
    lib = _lib.load()
    if _bound is lib:
        return lib
    i64, vp, sz, ci, cf = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
    for name, args in (("ss_glr_ckpt_bytes", [i64] * 3), ("ss_glr_workspace_bytes", [i64] * 3),
                       ("ss_glr_bwd_workspace_bytes", [i64] * 3 + [ci]), ("ss_glu_workspace_bytes", [i64] * 3 + [ci]),
                       ("ss_glu_bwd_workspace_bytes", [i64] * 3 + [ci]), ("ss_xent_workspace_bytes", [i64] * 3 + [ci]),
                       ("ss_xent_bwd_workspace_bytes", [i64] * 3 + [ci])):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, sz
    gates = [vp, i64, vp, i64, vp, i64, vp, cf]  # x, r, i with their row strides, decay, c
    for name, args in (("ss_glr_fwd", gates + [vp] * 6 + [sz] + [i64] * 3 + [ci, vp]),
                       ("ss_glr_bwd", gates + [vp] * 8 + [i64] + [vp] * 3 + [sz] + [i64] * 3 + [ci, vp]),
                       ("ss_glr_step", [vp] + gates + [vp] + [i64] * 2 + [ci, vp]),
                       ("ss_glu_fwd", [vp, i64, vp, vp, vp, ci, vp, sz] + [i64] * 3 + [ci, vp]),
                       ("ss_glu_bwd", [vp, i64] + [vp] * 6 + [ci, vp, sz] + [i64] * 3 + [ci, vp]),
                       ("ss_xent_fwd", [vp, i64, vp, vp, i64, vp, vp, vp, sz] + [i64] * 3 + [ci, vp]),
                       ("ss_xent_bwd", [vp, i64, vp, vp, i64, vp, vp, vp, vp, vp, sz] + [i64] * 3 + [ci, vp])):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, ci
    _bound = lib
    return lib
