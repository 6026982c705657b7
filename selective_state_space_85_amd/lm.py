"""torch-facing wrappers of the language-model operators (include/ss_lm.h): argument marshalling only.

Names and argument order follow the C entry points (``ss_glr_fwd`` -> ``glr_fwd``).  Every
operator runs in the HIP kernels of libssscan.so on torch's current stream.  As with the scan, the
results carry no autograd graph, also of tensors that require gradients: a forward and its backward
are joined in a ``torch.autograd.Function``, as ``examples/recurrent_lm.py`` does.
"""
from __future__ import annotations

import ctypes
from typing import Dict, Optional, Tuple, Union

import torch

from . import _lib, _lm
from .ops import _DTYPES
from .ops import _need as _refuse

_ACTS = {"silu": _lm.SS_ACT_SILU, "gelu": _lm.SS_ACT_GELU}
_BAD = ctypes.c_size_t(-1).value


def _p(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _code(dtype: torch.dtype) -> int:
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise TypeError("unsupported dtype %s" % dtype)
    return dt


def _dtype(t: torch.Tensor) -> int:
    return _code(t.dtype)


def _need(t: torch.Tensor, name: str, shape, dtype, device) -> None:
    """The checks of ``ops._need``, which words the refusal: these calls last a few microseconds."""
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        _refuse(t, name, shape, dtype, device)


def _gpu(t: torch.Tensor, fn: str) -> torch.device:
    if t.device.type != "cuda":
        raise ValueError("%s runs on the GPU; x is on %s" % (fn, t.device))
    return t.device


def _size(n: int) -> int:
    if n == _BAD:
        raise ValueError("invalid shape")
    return int(n)


def _space(need: int, workspace: Optional[torch.Tensor], device) -> Tuple[Optional[torch.Tensor], int]:
    """The caller's workspace, or one of `need` bytes (None if none is needed), and its size."""
    if workspace is None:
        return (torch.empty(need, dtype=torch.uint8, device=device), need) if need else (None, 0)
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on %s" % device)
    return workspace, workspace.numel() * workspace.element_size()


def _rows(t: torch.Tensor, name: str, shape, dtype, device) -> int:
    """Row stride of a tensor of `shape` whose rows have unit stride and lie evenly apart."""
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    n = shape[-1]
    if t.is_contiguous():
        return n
    st = t.stride()
    if len(shape) == 3:
        nb, nl = shape[0], shape[1]
        ld = st[1] if nl > 1 else (st[0] if nb > 1 else n)
        even = nb == 1 or nl == 1 or st[0] == nl * st[1]
    else:
        ld = st[0] if shape[0] > 1 else n
        even = True
    if not even or (n > 1 and st[-1] != 1) or ld < n:
        raise ValueError("%s rows must be evenly strided with unit inner stride" % name)
    return ld


# the current stream's handle: torch's own accessor of it, where there is one, takes a
# twentieth of the time of making a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class _on:
    """The tensor's device as the current one, and torch's current stream on it."""

    __slots__ = ("ctx", "stream")

    def __init__(self, device: torch.device):
        self.ctx = None if device.index == torch.cuda.current_device() else torch.cuda.device(device)
        self.stream = (_raw_stream(device.index) if _raw_stream is not None
                       else torch.cuda.current_stream(device).cuda_stream)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return self.stream

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _call(name: str, status: int) -> None:
    if status != _lib.SS_OK:
        _lib.check(name, status)


# ---------------------------------------------------------------- gated linear recurrence

def glr_ckpt_shape(batch: int, seqlen: int, dim: int) -> Tuple[int, int, int]:
    """Shape of the float32 kept states (``ss_glr_ckpt_bytes``): one every 32 rows."""
    _size(_lm.load().ss_glr_ckpt_bytes(batch, seqlen, dim))
    return (-(-seqlen // 32), batch, dim)


def glr_workspace_bytes(batch: int, seqlen: int, dim: int) -> int:
    """Workspace of ``ss_glr_fwd`` (0: none needed)."""
    return _size(_lm.load().ss_glr_workspace_bytes(batch, seqlen, dim))


def glr_bwd_workspace_bytes(batch: int, seqlen: int, dim: int, with_ckpt: bool = False) -> int:
    """Workspace of ``ss_glr_bwd``, with or without kept states given."""
    return _size(_lm.load().ss_glr_bwd_workspace_bytes(batch, seqlen, dim, int(with_ckpt)))


def _reset(reset: Optional[torch.Tensor], nb: int, nl: int, dev) -> Optional[torch.Tensor]:
    if reset is None:
        return None
    if reset.dtype not in (torch.bool, torch.uint8):
        raise TypeError("reset has dtype %s, expected bool or uint8" % reset.dtype)
    _need(reset, "reset", (nb, nl), reset.dtype, dev)
    return reset


def glr_fwd(x: torch.Tensor, r: torch.Tensor, i: torch.Tensor, decay: torch.Tensor, *, c: float = 8.0,
            h0: Optional[torch.Tensor] = None, reset: Optional[torch.Tensor] = None, return_last_state: bool = False,
            ckpt: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
            h_last: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """Gated linear recurrence ``ss_glr_fwd``:

        a_t = exp(-c softplus(decay) sigmoid(r_t)),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t

    x, r, i: (B, L, D), all float32 or all bfloat16, contiguous or column slices of a wider
    contiguous tensor; decay (D,) float32; h0 (B, D) float32; reset (B, L) bool or uint8, true
    where a new sequence starts.  ``ckpt``: a float32 tensor of ``glr_ckpt_shape`` that receives
    the states for ``glr_bwd``.  Returns y = h (B, L, D) and, if asked, h_last (B, D) float32.
    """
    if x.dim() != 3:
        raise ValueError("x must be (batch, seqlen, dim)")
    dev, dt, shape = _gpu(x, "glr_fwd"), _dtype(x), x.shape
    nb, nl, nd = shape
    lx, lr, li = (_rows(t, n, shape, x.dtype, dev) for t, n in ((x, "x"), (r, "r"), (i, "i")))
    _need(decay, "decay", (nd,), torch.float32, dev)
    if h0 is not None:
        _need(h0, "h0", (nb, nd), torch.float32, dev)
    reset = _reset(reset, nb, nl, dev)
    y = out if out is not None else x.new_empty(shape)
    _need(y, "out", shape, x.dtype, dev)
    if h_last is None and return_last_state:
        h_last = torch.empty((nb, nd), dtype=torch.float32, device=dev)
    if h_last is not None:
        _need(h_last, "h_last", (nb, nd), torch.float32, dev)
    if ckpt is not None:
        _need(ckpt, "ckpt", glr_ckpt_shape(nb, nl, nd), torch.float32, dev)
    ws, ws_bytes = _space(glr_workspace_bytes(nb, nl, nd), workspace, dev)
    with _on(dev) as stream:
        st = _lm.load().ss_glr_fwd(_p(x), lx, _p(r), lr, _p(i), li, _p(decay), c, _p(h0), _p(reset), _p(y), _p(h_last),
                                   _p(ckpt), _p(ws), ws_bytes, nb, nl, nd, dt, stream)
    _call("ss_glr_fwd", st)
    return (y, h_last) if return_last_state else y


def glr_bwd(x: torch.Tensor, r: torch.Tensor, i: torch.Tensor, decay: torch.Tensor, dy: torch.Tensor, *,
            c: float = 8.0, h0: Optional[torch.Tensor] = None, reset: Optional[torch.Tensor] = None,
            dh_last: Optional[torch.Tensor] = None, ckpt: Optional[torch.Tensor] = None, want_dh0: bool = True,
            out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """Gradients of sum(dy * y) + sum(dh_last * h_last) for ``glr_fwd`` with the same inputs
    (``ss_glr_bwd``).  With ``ckpt`` as ``glr_fwd`` wrote it the states are rebuilt from there,
    without it by a pass over the inputs.

    Returns a dict: dx, dr, di (B, L, D) in the input dtype, ddecay (D,) float32 and, if
    ``want_dh0``, dh0 (B, D) float32.  ``out``: a contiguous (B, L, 3 D) tensor that receives
    dx, dr and di side by side (the gradient of a joint projection); the dict then holds its slices.
    """
    if x.dim() != 3:
        raise ValueError("x must be (batch, seqlen, dim)")
    dev, dt, shape = _gpu(x, "glr_bwd"), _dtype(x), x.shape
    nb, nl, nd = shape
    lx, lr, li = (_rows(t, n, shape, x.dtype, dev) for t, n in ((x, "x"), (r, "r"), (i, "i")))
    _need(decay, "decay", (nd,), torch.float32, dev)
    _need(dy, "dy", shape, x.dtype, dev)
    for t, n in ((h0, "h0"), (dh_last, "dh_last")):
        if t is not None:
            _need(t, n, (nb, nd), torch.float32, dev)
    reset = _reset(reset, nb, nl, dev)
    if ckpt is not None:
        _need(ckpt, "ckpt", glr_ckpt_shape(nb, nl, nd), torch.float32, dev)
    if out is not None:
        _need(out, "out", (nb, nl, 3 * nd), x.dtype, dev)
        g = {"dx": out[..., :nd], "dr": out[..., nd:2 * nd], "di": out[..., 2 * nd:]}
        ld = 3 * nd
    else:
        g = {n: x.new_empty(shape) for n in ("dx", "dr", "di")}
        ld = nd
    g["ddecay"] = torch.empty((nd,), dtype=torch.float32, device=dev)
    if want_dh0:
        g["dh0"] = torch.empty((nb, nd), dtype=torch.float32, device=dev)
    ws, ws_bytes = _space(glr_bwd_workspace_bytes(nb, nl, nd, ckpt is not None), workspace, dev)
    with _on(dev) as stream:
        st = _lm.load().ss_glr_bwd(_p(x), lx, _p(r), lr, _p(i), li, _p(decay), c, _p(h0), _p(reset), _p(dy),
                                   _p(dh_last), _p(ckpt), _p(g["dx"]), _p(g["dr"]), _p(g["di"]), ld, _p(g["ddecay"]),
                                   _p(g.get("dh0")), _p(ws), ws_bytes, nb, nl, nd, dt, stream)
    _call("ss_glr_bwd", st)
    return g


def glr_step(h: torch.Tensor, x: torch.Tensor, r: torch.Tensor, i: torch.Tensor, decay: torch.Tensor, *,
             c: float = 8.0, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of the recurrence ``ss_glr_step``: h (B, D) float32 is updated in place.
    x, r, i: (B, D), contiguous or column slices of one wider tensor.  Returns y (B, D)."""
    if x.dim() != 2:
        raise ValueError("x must be (batch, dim)")
    dev, dt, shape = _gpu(x, "glr_step"), _dtype(x), x.shape
    nb, nd = shape
    lx = _rows(x, "x", shape, x.dtype, dev)
    lr = _rows(r, "r", shape, x.dtype, dev)
    li = _rows(i, "i", shape, x.dtype, dev)
    _need(h, "h", shape, torch.float32, dev)
    _need(decay, "decay", (nd,), torch.float32, dev)
    if out is None:
        out = x.new_empty(shape)
    else:
        _need(out, "out", shape, x.dtype, dev)
    with _on(dev) as stream:
        st = _lm.load().ss_glr_step(_p(h), _p(x), lx, _p(r), lr, _p(i), li, _p(decay), c, _p(out), nb, nd, dt, stream)
    _call("ss_glr_step", st)
    return out


# ---------------------------------------------------------------- gated feed-forward projection

def glu_workspace_bytes(tokens: int, dim: int, features: int, dtype: torch.dtype) -> int:
    """Workspace of ``ss_glu_fwd`` (0: none needed)."""
    return _size(_lm.load().ss_glu_workspace_bytes(tokens, dim, features, _code(dtype)))


def glu_bwd_workspace_bytes(tokens: int, dim: int, features: int, dtype: torch.dtype) -> int:
    """Workspace of ``ss_glu_bwd``."""
    return _size(_lm.load().ss_glu_bwd_workspace_bytes(tokens, dim, features, _code(dtype)))


def _tokens(x: torch.Tensor, fn: str) -> Tuple[int, int, int]:
    """(tokens, dim, row stride) of an operand (..., dim) whose tokens lie evenly apart."""
    if x.dim() < 2 or x.dim() > 3:
        raise ValueError("%s: x must be (tokens, dim) or (batch, seqlen, dim)" % fn)
    ld = _rows(x, "x", x.shape, x.dtype, x.device)
    n = 1
    for s in x.shape[:-1]:
        n *= s
    return n, x.shape[-1], ld


def _act(act: str) -> int:
    if act not in _ACTS:
        raise ValueError("act must be one of %s, not %r" % (", ".join(sorted(_ACTS)), act))
    return _ACTS[act]


def glu_fwd(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, *, act: str = "silu",
            out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gated feed-forward projection ``ss_glu_fwd``: h = act(x w_gate^T) * (x w_up^T) in one kernel.

    x (..., K) with one or two leading axes, contiguous or a column slice; w_gate, w_up (F, K);
    all float32 or all bfloat16.  act: "silu" or "gelu" (tanh form).  Returns h (..., F)."""
    dev, dt = _gpu(x, "glu_fwd"), _dtype(x)
    m, k, ld = _tokens(x, "glu_fwd")
    f = w_gate.shape[0]
    _need(w_gate, "w_gate", (f, k), x.dtype, dev)
    _need(w_up, "w_up", (f, k), x.dtype, dev)
    shape = x.shape[:-1] + (f,)
    if out is None:
        out = x.new_empty(shape)
    else:
        _need(out, "out", shape, x.dtype, dev)
    lib = _lm.load()
    ws, ws_bytes = _space(_size(lib.ss_glu_workspace_bytes(m, k, f, dt)), workspace, dev)
    with _on(dev) as stream:
        st = lib.ss_glu_fwd(_p(x), ld, _p(w_gate), _p(w_up), _p(out), _act(act), _p(ws), ws_bytes, m, k, f, dt, stream)
    _call("ss_glu_fwd", st)
    return out


def glu_bwd(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, dh: torch.Tensor, *, act: str = "silu",
            want_dx: bool = True, want_dw: bool = True,
            workspace: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """Gradients of sum(dh * h) for ``glu_fwd`` with the same inputs (``ss_glu_bwd``): a dict of
    dx (..., K) and dw_gate, dw_up (F, K), those that are wanted, in the input dtype."""
    dev, dt = _gpu(x, "glu_bwd"), _dtype(x)
    m, k, ld = _tokens(x, "glu_bwd")
    f = w_gate.shape[0]
    _need(w_gate, "w_gate", (f, k), x.dtype, dev)
    _need(w_up, "w_up", (f, k), x.dtype, dev)
    _need(dh, "dh", x.shape[:-1] + (f,), x.dtype, dev)
    g = {}
    if want_dx:
        g["dx"] = x.new_empty(x.shape)
    if want_dw:
        g["dw_gate"] = x.new_empty((f, k))
        g["dw_up"] = x.new_empty((f, k))
    lib = _lm.load()
    ws, ws_bytes = _space(_size(lib.ss_glu_bwd_workspace_bytes(m, k, f, dt)), workspace, dev)
    with _on(dev) as stream:
        st = lib.ss_glu_bwd(_p(x), ld, _p(w_gate), _p(w_up), _p(dh), _p(g.get("dx")), _p(g.get("dw_gate")),
                            _p(g.get("dw_up")), _act(act), _p(ws), ws_bytes, m, k, f, dt, stream)
    _call("ss_glu_bwd", st)
    return g


# ---------------------------------------------------------------- vocabulary cross entropy

def xent_workspace_bytes(tokens: int, dim: int, vocab: int, dtype: torch.dtype) -> int:
    """Workspace of ``ss_xent_fwd``."""
    return _size(_lm.load().ss_xent_workspace_bytes(tokens, dim, vocab, _code(dtype)))


def xent_bwd_workspace_bytes(tokens: int, dim: int, vocab: int, dtype: torch.dtype) -> int:
    """Workspace of ``ss_xent_bwd``."""
    return _size(_lm.load().ss_xent_bwd_workspace_bytes(tokens, dim, vocab, _code(dtype)))


def xent_fwd(x: torch.Tensor, w: torch.Tensor, target: torch.Tensor, *, ignore_index: int = -100,
             workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Softmax cross entropy of the logits x w^T, which are not stored (``ss_xent_fwd``).

    x (..., K) with one or two leading axes, contiguous or a column slice; w (V, K); both
    float32 or both bfloat16; target (...,) int64.  Returns (loss, lse), float32 of target's
    shape: loss = lse - logit[target], 0 where the target is ignore_index or outside [0, V)."""
    dev, dt = _gpu(x, "xent_fwd"), _dtype(x)
    n, k, ld = _tokens(x, "xent_fwd")
    v = w.shape[0]
    _need(w, "w", (v, k), x.dtype, dev)
    _need(target, "target", x.shape[:-1], torch.int64, dev)
    loss = torch.empty(target.shape, dtype=torch.float32, device=dev)
    lse = torch.empty(target.shape, dtype=torch.float32, device=dev)
    lib = _lm.load()
    ws, ws_bytes = _space(_size(lib.ss_xent_workspace_bytes(n, k, v, dt)), workspace, dev)
    with _on(dev) as stream:
        st = lib.ss_xent_fwd(_p(x), ld, _p(w), _p(target), ignore_index, _p(loss), _p(lse), _p(ws), ws_bytes, n, k, v,
                             dt, stream)
    _call("ss_xent_fwd", st)
    return loss, lse


def xent_bwd(x: torch.Tensor, w: torch.Tensor, target: torch.Tensor, lse: torch.Tensor, dloss: torch.Tensor, *,
             ignore_index: int = -100, want_dx: bool = True, want_dw: bool = True,
             workspace: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """Gradients of sum(dloss * loss) for ``xent_fwd`` with the same inputs and its lse
    (``ss_xent_bwd``): a dict of dx (..., K) and dw (V, K), those that are wanted, in the
    input dtype.  dloss: float32 of target's shape."""
    dev, dt = _gpu(x, "xent_bwd"), _dtype(x)
    n, k, ld = _tokens(x, "xent_bwd")
    v = w.shape[0]
    _need(w, "w", (v, k), x.dtype, dev)
    _need(target, "target", x.shape[:-1], torch.int64, dev)
    _need(lse, "lse", target.shape, torch.float32, dev)
    _need(dloss, "dloss", target.shape, torch.float32, dev)
    g = {}
    if want_dx:
        g["dx"] = x.new_empty(x.shape)
    if want_dw:
        g["dw"] = x.new_empty((v, k))
    lib = _lm.load()
    ws, ws_bytes = _space(_size(lib.ss_xent_bwd_workspace_bytes(n, k, v, dt)), workspace, dev)
    with _on(dev) as stream:
        st = lib.ss_xent_bwd(_p(x), ld, _p(w), _p(target), ignore_index, _p(lse), _p(dloss), _p(g.get("dx")),
                             _p(g.get("dw")), _p(ws), ws_bytes, n, k, v, dt, stream)
    _call("ss_xent_bwd", st)
    return g
