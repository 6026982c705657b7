"""Plain float64 NumPy statements of the language-model operators (include/ss_lm.h), token by
token and element by element as the header defines them, with their gradients by the chain
rule.  Test infrastructure only."""
import numpy as np


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def _rates(decay, c):
    return c * np.logaddexp(0.0, decay)


def _gates(r, k, reset_t):
    s = sigmoid(r)
    a = np.exp(-k * s)
    m = np.sqrt(-np.expm1(-2.0 * k * s))
    if reset_t is not None:
        on = reset_t[:, None] != 0
        a, m = np.where(on, 0.0, a), np.where(on, 1.0, m)
    return a, m, s


def glr(x, r, i, decay, c, h0=None, reset=None):
    """(y, h_last); x, r, i (B, L, D) float64."""
    nb, nl, nd = x.shape
    k = _rates(decay, c)
    h = np.zeros((nb, nd)) if h0 is None else h0.astype(np.float64)
    y = np.empty((nb, nl, nd))
    for t in range(nl):
        a, m, _ = _gates(r[:, t], k, None if reset is None else reset[:, t])
        h = a * h + m * sigmoid(i[:, t]) * x[:, t]
        y[:, t] = h
    return y, h


def glr_bwd(x, r, i, decay, c, dy, h0=None, reset=None, dh_last=None):
    nb, nl, nd = x.shape
    k = _rates(decay, c)
    y, _ = glr(x, r, i, decay, c, h0, reset)
    first = np.zeros((nb, nd)) if h0 is None else h0.astype(np.float64)
    g = np.zeros((nb, nd)) if dh_last is None else dh_last.astype(np.float64)
    dx, dr, di = np.empty_like(x), np.empty_like(x), np.empty_like(x)
    dk = np.zeros(nd)
    for t in range(nl - 1, -1, -1):
        g = g + dy[:, t]
        a, m, s = _gates(r[:, t], k, None if reset is None else reset[:, t])
        si = sigmoid(i[:, t])
        before = y[:, t - 1] if t > 0 else first
        with np.errstate(divide="ignore", invalid="ignore"):
            # d m / d log a = -a^2 / m, times ds/dr = s (1 - s): 0 where the gate is shut (m = 0)
            slope = np.where(m > 0, -a * a / m, 0.0)
        dla = g * (a * before + slope * si * x[:, t])
        dx[:, t] = g * m * si
        di[:, t] = g * m * x[:, t] * si * (1.0 - si)
        dr[:, t] = -k * dla * s * (1.0 - s)
        dk -= (dla * s).sum(0)
        g = a * g
    return {"dx": dx, "dr": dr, "di": di, "ddecay": dk * c * sigmoid(decay), "dh0": g}


def _act(g, act):
    if act == "silu":
        s = sigmoid(g)
        return g * s, s * (1.0 + g * (1.0 - s))
    q = np.sqrt(2.0 / np.pi)
    th = np.tanh(q * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th ** 2) * q * (1.0 + 3 * 0.044715 * g ** 2)


def glu(x, wg, wu, act):
    g, u = x @ wg.T, x @ wu.T
    return _act(g, act)[0] * u


def glu_bwd(x, wg, wu, dh, act):
    g, u = x @ wg.T, x @ wu.T
    f, slope = _act(g, act)
    dg, du = dh * u * slope, dh * f
    return {"dx": dg @ wg + du @ wu, "dw_gate": dg.T @ x, "dw_up": du.T @ x}


def xent(x, w, target, ignore=-100):
    """(loss, lse, logits)"""
    l = x @ w.T
    top = l.max(1, keepdims=True)
    lse = (top + np.log(np.exp(l - top).sum(1, keepdims=True)))[:, 0]
    live = (target != ignore) & (target >= 0) & (target < w.shape[0])
    loss = np.where(live, lse - l[np.arange(len(l)), np.where(live, target, 0)], 0.0)
    return loss, lse, l, live


def xent_bwd(x, w, target, dloss, ignore=-100):
    _, lse, l, live = xent(x, w, target, ignore)
    p = np.exp(l - lse[:, None])
    p[np.arange(len(l)), np.where(live, target, 0)] -= 1.0
    p *= np.where(live, dloss, 0.0)[:, None]
    return {"dx": p @ w, "dw": p.T @ x}
