"""Plain float64 NumPy statements of the linear-attention operators and of sampling
(include/ss_attn.h), token by token as the header defines them, with their gradients by the
chain rule.  Test infrastructure only."""
import numpy as np


def _spread(x, h):
    """Heads that share queries and keys side by side."""
    return np.repeat(x, h // x.shape[-2], axis=-2)


def lattn(q, k, v, log_decay, scale, h0=None, reset=None):
    """(o, h_last); q, k (B, L, Hk, K), v (B, L, H, V) float64."""
    nb, nl, nh, dv = v.shape
    q, k = _spread(q, nh), _spread(k, nh)
    a = np.exp(log_decay)[None, :, None, None]
    st = np.zeros((nb, nh, q.shape[-1], dv)) if h0 is None else h0.astype(np.float64)
    o = np.empty(v.shape)
    for t in range(nl):
        st = a * st
        if reset is not None:
            st = np.where((reset[:, t] != 0)[:, None, None, None], 0.0, st)
        st = st + k[:, t, :, :, None] * v[:, t, :, None, :]
        o[:, t] = scale * (q[:, t, :, :, None] * st).sum(2)
    return o, st


def lattn_bwd(q, k, v, log_decay, scale, do, h0=None, reset=None, dh_last=None):
    nb, nl, nh, dv = v.shape
    share = nh // q.shape[2]
    qs, ks = _spread(q, nh), _spread(k, nh)
    a = np.exp(log_decay)[None, :, None, None]
    keep = np.ones((nb, nl)) if reset is None else (reset == 0).astype(np.float64)
    st = np.zeros((nb, nh, q.shape[-1], dv)) if h0 is None else h0.astype(np.float64)
    dq, dk, dvv = np.empty(qs.shape), np.empty(qs.shape), np.empty(v.shape)
    for t in range(nl):
        st = np.where(keep[:, t, None, None, None] != 0, a * st, 0.0) + ks[:, t, :, :, None] * v[:, t, :, None, :]
        dq[:, t] = scale * (st * do[:, t, :, None, :]).sum(-1)
    g = np.zeros_like(st) if dh_last is None else dh_last.astype(np.float64)
    for t in range(nl - 1, -1, -1):
        g = g + scale * qs[:, t, :, :, None] * do[:, t, :, None, :]
        dk[:, t] = (g * v[:, t, :, None, :]).sum(-1)
        dvv[:, t] = (g * ks[:, t, :, :, None]).sum(2)
        g = np.where(keep[:, t, None, None, None] != 0, a * g, 0.0)
    shape = q.shape[:3] + (share, q.shape[-1])
    return {"dq": dq.reshape(shape).sum(3), "dk": dk.reshape(shape).sum(3), "dv": dvv, "dh0": g}


def _turn(y, pos, inv_freq, interleaved, sign=1.0):
    n = len(inv_freq)
    ang = pos[..., None, None].astype(np.float64) * inv_freq.astype(np.float64)
    c, s = np.cos(ang), sign * np.sin(ang)
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    out = y.copy()
    out[..., i] = y[..., i] * c - y[..., j] * s
    out[..., j] = y[..., j] * c + y[..., i] * s
    return out


def qknorm(x, w, pos, inv_freq, eps, interleaved):
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return _turn(x * r * w, pos, inv_freq, interleaved)


def qknorm_bwd(x, w, pos, inv_freq, eps, interleaved, dy):
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g = _turn(dy, pos, inv_freq, interleaved, -1.0)
    xr = x * r
    return r * (g * w - xr * (g * w * xr).mean(-1, keepdims=True)), (g * xr).reshape(-1, x.shape[-1]).sum(0)


def sample_row(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The token of one row; every argument a float64 that holds the float32 the call was given."""
    index = np.arange(len(logits))
    can = logits > -np.inf  # NaN compares false
    if not can.any():
        return -1
    order = index[can][np.argsort(-logits[can], kind="stable")]
    if not temperature > 0:
        return int(order[0])
    l = logits[order]
    with np.errstate(invalid="ignore", over="ignore"):
        w = (l == np.inf).astype(np.float64) if l[0] == np.inf else np.exp((l - l[0]) / temperature)
    # the fixed point that weights are rounded to, of the largest's: tokens below half a unit have none
    unit = 2.0 ** min(50, 62 - len(logits).bit_length())
    w = np.rint(w * unit) / unit
    if top_k > 0:
        order, w = order[:top_k], w[:top_k]
    if top_p < 1:
        before = np.cumsum(w) - w
        n = max(1, int((before < top_p * w.sum()).sum()))
        order, w = order[:n], w[:n]
    if min_p > 0:
        n = max(1, int((w >= min_p).sum()))
        order, w = order[:n], w[:n]
    total = np.cumsum(w)
    at = int(np.searchsorted(total, (u if u > 0 else 0.0) * total[-1], side="right"))
    return int(order[min(at, int(np.flatnonzero(w)[-1]))])
