"""torch-facing wrappers of linear attention, of the norms of its queries and keys, and of sampling
(include/ss_attn.h): argument marshalling only.

Names and argument order follow the C entry points (``ss_lattn_fwd`` -> ``lattn_fwd``).  Every
operator runs in the HIP kernels of libssscan.so on torch's current stream.  As with the scan, the
results carry no autograd graph: a forward and its backward are joined in a
``torch.autograd.Function``, as ``examples/recurrent_lm.py`` does.
"""
from __future__ import annotations

from typing import Dict, Optional, Tuple, Union

import torch

from . import _attn
from .lm import _call, _code, _dtype, _gpu, _need, _on, _p, _size, _space


def _heads(t: torch.Tensor, name: str, shape, dtype, device) -> int:
    """Token stride of a tensor (tokens..., heads, width) whose heads lie side by side and whose
    tokens lie evenly apart."""
    if t.shape == shape and t.dtype == dtype and t.device == device and t.is_contiguous():
        return shape[-2] * shape[-1]
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    h, w = shape[-2], shape[-1]
    st = t.stride()
    row = (w == 1 or st[-1] == 1) and (h == 1 or st[-2] == w)
    if len(shape) == 4:
        nb, nl = shape[0], shape[1]
        ld = st[1] if nl > 1 else (st[0] if nb > 1 else h * w)
        even = nb == 1 or nl == 1 or st[0] == nl * st[1]
    else:
        ld = st[0] if shape[0] > 1 else h * w
        even = True
    if not (row and even) or ld < h * w:
        raise ValueError("%s must hold its heads side by side in evenly strided rows" % name)
    return ld


def _shared(qk_heads: int, heads: int) -> None:
    if qk_heads == 0 or heads % qk_heads != 0:
        raise ValueError("v's %d heads are not a multiple of q's %d" % (heads, qk_heads))


def _scale(scale: Optional[float], k_dim: int) -> float:
    """The one given, or k_dim ** -0.5 (heads without a width have none; the library refuses them)."""
    return scale if scale is not None else k_dim ** -0.5 if k_dim else 1.0


def _like(t: torch.Tensor) -> torch.Tensor:
    """A contiguous result of t's shape and type."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _flags(reset: Optional[torch.Tensor], shape, dev) -> None:
    if reset is not None:
        if reset.dtype not in (torch.bool, torch.uint8):
            raise TypeError("reset has dtype %s, expected bool or uint8" % reset.dtype)
        _need(reset, "reset", shape, reset.dtype, dev)


# ---------------------------------------------------------------- linear attention

def lattn_workspace_bytes(batch: int, seqlen: int, qk_heads: int, heads: int, k_dim: int, v_dim: int,
                          dtype: torch.dtype) -> int:
    """Workspace of ``ss_lattn_fwd`` (0: none needed)."""
    return _size(_attn.load().ss_lattn_workspace_bytes(batch, seqlen, qk_heads, heads, k_dim, v_dim, _code(dtype)))


def lattn_bwd_workspace_bytes(batch: int, seqlen: int, qk_heads: int, heads: int, k_dim: int, v_dim: int,
                              dtype: torch.dtype) -> int:
    """Workspace of ``ss_lattn_bwd`` (0: none needed)."""
    return _size(_attn.load().ss_lattn_bwd_workspace_bytes(batch, seqlen, qk_heads, heads, k_dim, v_dim, _code(dtype)))


def _attention(q, k, v, log_decay, scale, h0, reset, fn):
    """The checks that the forward and the backward share: device, type code, sizes and row strides."""
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("%s: q, k and v must be (batch, seqlen, heads, width)" % fn)
    dev, dt = _gpu(q, fn), _dtype(q)
    shape, dtype = q.shape, q.dtype
    nb, nl, hk, dk = shape
    nh, dv = v.shape[2], v.shape[3]
    _shared(hk, nh)
    lds = (_heads(q, "q", shape, dtype, dev), _heads(k, "k", shape, dtype, dev), _heads(v, "v", (nb, nl, nh, dv), dtype, dev))
    _need(log_decay, "log_decay", (nh,), torch.float32, dev)
    if h0 is not None:
        _need(h0, "h0", (nb, nh, dk, dv), torch.float32, dev)
    _flags(reset, (nb, nl), dev)
    return dev, dt, (nb, nl, hk, nh, dk, dv), lds, _scale(scale, dk)


def lattn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, *,
              scale: Optional[float] = None, h0: Optional[torch.Tensor] = None,
              reset: Optional[torch.Tensor] = None, return_last_state: bool = False,
              out: Optional[torch.Tensor] = None, h_last: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """Linear attention with a decay for each head ``ss_lattn_fwd``:

        S_t = exp(log_decay) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t

    q, k: (B, L, Hk, K); v: (B, L, H, V), H a multiple of Hk (heads that share queries and keys lie
    side by side); all float32 or all bfloat16, contiguous or slices of a wider tensor's rows.
    log_decay (H,) float32, at most 0; scale: K ** -0.5 by default; h0 (B, H, K, V) float32; reset
    (B, L) bool or uint8, true where a new sequence starts.  K and V are at most 256.  Returns
    o (B, L, H, V) and, if asked, the state after the last row (B, H, K, V) float32 (``h_last``, which
    may be h0 itself)."""
    dev, dt, (nb, nl, hk, nh, dk, dv), (lq, lk, lv), scale = _attention(q, k, v, log_decay, scale, h0, reset, "lattn_fwd")
    if out is None:
        out = _like(v)
    else:
        _need(out, "out", (nb, nl, nh, dv), q.dtype, dev)
    if h_last is None and return_last_state:
        h_last = torch.empty((nb, nh, dk, dv), dtype=torch.float32, device=dev)
    if h_last is not None:
        _need(h_last, "h_last", (nb, nh, dk, dv), torch.float32, dev)
    lib = _attn.load()
    ws, ws_bytes = _space(_size(lib.ss_lattn_workspace_bytes(nb, nl, hk, nh, dk, dv, dt)), workspace, dev)
    with _on(dev) as stream:
        st = lib.ss_lattn_fwd(_p(q), lq, _p(k), lk, _p(v), lv, _p(log_decay), scale, _p(h0), _p(reset), _p(out),
                              _p(h_last), _p(ws), ws_bytes, nb, nl, hk, nh, dk, dv, dt, stream)
    _call("ss_lattn_fwd", st)
    return (out, h_last) if return_last_state else out


def lattn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, do: torch.Tensor, *,
              scale: Optional[float] = None, h0: Optional[torch.Tensor] = None, reset: Optional[torch.Tensor] = None,
              dh_last: Optional[torch.Tensor] = None, want_dh0: bool = False,
              workspace: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """Gradients of sum(do * o) + sum(dh_last * h_last) for ``lattn_fwd`` with the same inputs
    (``ss_lattn_bwd``): a dict of dq, dk (B, L, Hk, K), dv (B, L, H, V) in the input dtype and, if
    ``want_dh0``, dh0 (B, H, K, V) float32.  do: (B, L, H, V), strided as v may be.  log_decay is a
    constant of the layer and has no gradient."""
    dev, dt, (nb, nl, hk, nh, dk, dv), (lq, lk, lv), scale = _attention(q, k, v, log_decay, scale, h0, reset, "lattn_bwd")
    ldo = _heads(do, "do", (nb, nl, nh, dv), q.dtype, dev)
    if dh_last is not None:
        _need(dh_last, "dh_last", (nb, nh, dk, dv), torch.float32, dev)
    g = {"dq": _like(q), "dk": _like(k), "dv": _like(v)}
    if want_dh0:
        g["dh0"] = torch.empty((nb, nh, dk, dv), dtype=torch.float32, device=dev)
    lib = _attn.load()
    ws, ws_bytes = _space(_size(lib.ss_lattn_bwd_workspace_bytes(nb, nl, hk, nh, dk, dv, dt)), workspace, dev)
    with _on(dev) as stream:
        st = lib.ss_lattn_bwd(_p(q), lq, _p(k), lk, _p(v), lv, _p(log_decay), scale, _p(h0), _p(reset), _p(do), ldo,
                              _p(dh_last), _p(g["dq"]), _p(g["dk"]), _p(g["dv"]), _p(g.get("dh0")), _p(ws), ws_bytes,
                              nb, nl, hk, nh, dk, dv, dt, stream)
    _call("ss_lattn_bwd", st)
    return g


def lattn_step(h: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, *,
               scale: Optional[float] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of the recurrence ``ss_lattn_step``: h (B, H, K, V) float32 is updated in place.
    q, k: (B, Hk, K); v: (B, H, V), contiguous or slices of a wider tensor's rows.  Returns o (B, H, V)."""
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("lattn_step: q, k and v must be (batch, heads, width)")
    dev, dt = _gpu(q, "lattn_step"), _dtype(q)
    shape, dtype = q.shape, q.dtype
    nb, hk, dk = shape
    nh, dv = v.shape[1], v.shape[2]
    _shared(hk, nh)
    lq = _heads(q, "q", shape, dtype, dev)
    lk = _heads(k, "k", shape, dtype, dev)
    lv = _heads(v, "v", (nb, nh, dv), dtype, dev)
    _need(h, "h", (nb, nh, dk, dv), torch.float32, dev)
    _need(log_decay, "log_decay", (nh,), torch.float32, dev)
    if out is None:
        out = _like(v)
    else:
        _need(out, "out", (nb, nh, dv), dtype, dev)
    with _on(dev) as stream:
        st = _attn.load().ss_lattn_step(_p(h), _p(q), lq, _p(k), lk, _p(v), lv, _p(log_decay),
                                        _scale(scale, dk), _p(out), nb, hk, nh, dk, dv, dt, stream)
    _call("ss_lattn_step", st)
    return out


# ---------------------------------------------------------------- norms and rotation of queries and keys

def qknorm_bwd_workspace_bytes(tokens: int, q_heads: int, k_heads: int, width: int) -> int:
    """Workspace of ``ss_qknorm_bwd``."""
    return _size(_attn.load().ss_qknorm_bwd_workspace_bytes(tokens, q_heads, k_heads, width))


def _norm(q, k, w_q, w_k, pos, inv_freq, fn):
    """The checks of both directions: device, type code, sizes and row strides."""
    shape, dtype = q.shape, q.dtype
    if len(shape) == 4:
        nb, nl, hq, width = shape
        lead, n = (nb, nl), nb * nl
    elif len(shape) == 3:
        n, hq, width = shape
        lead = (n,)
    if len(shape) not in (3, 4) or k.dim() != len(shape):
        raise ValueError("%s: q and k must be (tokens, heads, width) or (batch, seqlen, heads, width)" % fn)
    dev, dt = _gpu(q, fn), _code(dtype)
    hk = k.shape[-2]
    lq = _heads(q, "q", shape, dtype, dev)
    lk = _heads(k, "k", lead + (hk, width), dtype, dev)
    _need(w_q, "w_q", (width,), torch.float32, dev)
    _need(w_k, "w_k", (width,), torch.float32, dev)
    _need(pos, "pos", lead, torch.int64, dev)
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must have one axis")
    half = inv_freq.shape[0]
    _need(inv_freq, "inv_freq", (half,), torch.float32, dev)
    return dev, dt, lq, lk, (n, hq, hk, width, half)


def qknorm_fwd(q: torch.Tensor, k: torch.Tensor, w_q: torch.Tensor, w_k: torch.Tensor, pos: torch.Tensor,
               inv_freq: torch.Tensor, *, eps: float = 1e-6, interleaved: bool = False,
               out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Norms of queries and keys for each head, and their position rotation ``ss_qknorm_fwd``:

        y = x / sqrt(mean(x^2) + eps) * w,  pair i of y's first 2 n elements turned by pos * inv_freq[i]

    q (..., Hq, W) and k (..., Hk, W) with one or two leading axes, both float32 or both bfloat16,
    contiguous or slices of a wider tensor's rows; w_q, w_k (W,) float32; pos (...,) int64; inv_freq
    (n,) float32, n at most W / 2 (n = 0: norms alone).  Pairs are (i, i + n), or (2 i, 2 i + 1) with
    ``interleaved``.  ``out``: contiguous tensors of q's and k's shapes.  Returns (qo, ko)."""
    dev, dt, lq, lk, sizes = _norm(q, k, w_q, w_k, pos, inv_freq, "qknorm_fwd")
    qo, ko = (_like(q), _like(k)) if out is None else out
    if out is not None:
        _need(qo, "out[0]", q.shape, q.dtype, dev)
        _need(ko, "out[1]", k.shape, q.dtype, dev)
    with _on(dev) as stream:
        st = _attn.load().ss_qknorm_fwd(_p(q), lq, _p(k), lk, _p(w_q), _p(w_k), _p(pos), _p(inv_freq), eps,
                                        int(interleaved), _p(qo), _p(ko), *sizes, dt, stream)
    _call("ss_qknorm_fwd", st)
    return qo, ko


def qknorm_bwd(q: torch.Tensor, k: torch.Tensor, w_q: torch.Tensor, w_k: torch.Tensor, pos: torch.Tensor,
               inv_freq: torch.Tensor, dqo: torch.Tensor, dko: torch.Tensor, *, eps: float = 1e-6,
               interleaved: bool = False, workspace: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """Gradients of sum(dqo * qo) + sum(dko * ko) for ``qknorm_fwd`` with the same inputs
    (``ss_qknorm_bwd``): a dict of dq, dk in the input dtype and dw_q, dw_k (W,) float32."""
    dev, dt, lq, lk, sizes = _norm(q, k, w_q, w_k, pos, inv_freq, "qknorm_bwd")
    _need(dqo, "dqo", q.shape, q.dtype, dev)
    _need(dko, "dko", k.shape, q.dtype, dev)
    g = {"dq": _like(q), "dk": _like(k),
         "dw_q": torch.empty(w_q.shape, dtype=torch.float32, device=dev),
         "dw_k": torch.empty(w_k.shape, dtype=torch.float32, device=dev)}
    lib = _attn.load()
    ws, ws_bytes = _space(_size(lib.ss_qknorm_bwd_workspace_bytes(*sizes[:4])), workspace, dev)
    with _on(dev) as stream:
        st = lib.ss_qknorm_bwd(_p(q), lq, _p(k), lk, _p(w_q), _p(w_k), _p(pos), _p(inv_freq), eps, int(interleaved),
                               _p(dqo), _p(dko), _p(g["dq"]), _p(g["dk"]), _p(g["dw_q"]), _p(g["dw_k"]), _p(ws),
                               ws_bytes, *sizes, dt, stream)
    _call("ss_qknorm_bwd", st)
    return g


# ---------------------------------------------------------------- sampling

def sample_workspace_bytes(rows: int, vocab: int, dtype: torch.dtype) -> int:
    """Workspace of ``ss_sample`` (0: none needed)."""
    return _size(_attn.load().ss_sample_workspace_bytes(rows, vocab, _code(dtype)))


def _setting(v, name: str, rows: int, dtype, device):
    """(tensor or None, value for all rows)"""
    if isinstance(v, torch.Tensor):
        _need(v, name, (rows,), dtype, device)
        return v, 0
    return None, v


def sample(logits: torch.Tensor, u: torch.Tensor, *, temperature: Union[float, torch.Tensor] = 1.0,
           top_k: Union[int, torch.Tensor] = 0, top_p: Union[float, torch.Tensor] = 1.0,
           min_p: Union[float, torch.Tensor] = 0.0, out: Optional[torch.Tensor] = None,
           workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token for each row of logits from one given random number ``ss_sample``.

    logits (rows, V) float32 or bfloat16, rows evenly strided; u (rows,) float32 in [0, 1).  Of the
    tokens in falling order of their logits (equal ones by index), with weights
    exp((l - largest) / temperature), the first top_k remain (0: all), of these the ones before which the
    weights sum to less than top_p of their sum, and of these the ones with weight at least min_p; the
    token is the first at which the running sum exceeds u times the sum.  The settings are numbers, or
    (rows,) tensors: float32, top_k int32.  A temperature of 0 takes the largest logit; NaN and -infinity
    are never taken (-1: a row of nothing else).  Returns (rows,) int64."""
    if logits.dim() != 2:
        raise ValueError("logits must be (rows, vocab)")
    dev, dt = _gpu(logits, "sample"), _dtype(logits)
    n, v = logits.shape
    if (v > 1 and logits.stride(1) != 1) or (n > 1 and logits.stride(0) < v):
        raise ValueError("logits rows must be evenly strided with unit inner stride")
    ld = logits.stride(0) if n > 1 else v
    _need(u, "u", (n,), torch.float32, dev)
    t, t_all = _setting(temperature, "temperature", n, torch.float32, dev)
    k, k_all = _setting(top_k, "top_k", n, torch.int32, dev)
    p, p_all = _setting(top_p, "top_p", n, torch.float32, dev)
    m, m_all = _setting(min_p, "min_p", n, torch.float32, dev)
    k_all = max(0, min(int(k_all), 2 ** 31 - 1))
    if out is None:
        out = torch.empty((n,), dtype=torch.int64, device=dev)
    else:
        _need(out, "out", (n,), torch.int64, dev)
    lib = _attn.load()
    ws, ws_bytes = _space(_size(lib.ss_sample_workspace_bytes(n, v, dt)), workspace, dev)
    with _on(dev) as stream:
        st = lib.ss_sample(_p(logits), ld, _p(u), _p(t), t_all, _p(k), k_all, _p(p), p_all, _p(m), m_all, _p(out),
                           _p(ws), ws_bytes, n, v, dt, stream)
    _call("ss_sample", st)
    return out
