"""Cases, plain forms and 64-bit definitions of the operators of a layer that mixes tokens by linear
attention, and of the choice of the next token:

* linear attention with a decay for each head (``lattn_fwd``, ``lattn_bwd``, ``lattn_step``),
* the norms of its queries and keys with their position rotation (``qknorm_fwd``, ``qknorm_bwd``),
* sampling from logits with temperature, top-k, top-p and min-p (``sample``).

With ``own`` false, ``run`` computes each in elementary torch operations in 32 bits (angles, and
sampling's weights and their sums, in 64), rounded once at the end; with ``own`` true it makes the
library's calls.
"""
import math

import numpy as np
import torch

own = False

F32, BF16 = "f32", "bf16"
ROPE_BASE = 10000.0
EPS = 1e-6


# ---------------------------------------------------------------------------------- the cases

def listed():
    return [
        # serving, one sequence: one token through one layer's heads (latency only)
        dict(name="lattn-step-one", op="lattn_step", dtype=BF16, b=1, l=1, hk=20, h=20, dk=128, dv=128),
        # serving, a full batch: one token of 256 sequences, the states read and written once
        dict(name="lattn-step-batch", op="lattn_step", dtype=BF16, b=256, l=1, hk=40, h=40, dk=128, dv=128),
        # serving, a long prompt: one sequence of the long context, its state kept for decoding
        dict(name="lattn-prompt-long", op="lattn_prompt", dtype=BF16, b=1, l=131072, hk=16, h=16, dk=128, dv=128),
        # training, the large-model layer: forward, then every gradient
        dict(name="lattn-train-large", op="lattn_train", dtype=BF16, b=8, l=2048, hk=40, h=40, dk=128, dv=128,
             packed=False),
        # training on packed documents of odd sizes in 32 bits, queries and keys shared by three
        # heads of values each, continued from a state
        dict(name="lattn-train-packed", op="lattn_train", dtype=F32, b=3, l=1021, hk=4, h=12, dk=72, dv=91,
             packed=True),
        # serving, one sequence: the queries and keys of one token far into its context
        dict(name="qknorm-token", op="qknorm_fwd", dtype=BF16, b=1, l=1, hq=20, hk=20, d=128, rot=128, inter=False,
             far=131071),
        # serving, a long prompt with keys shared by four heads, half of each head rotated
        dict(name="qknorm-prompt", op="qknorm_fwd", dtype=BF16, b=1, l=131072, hq=16, hk=4, d=128, rot=64, inter=True,
             far=0),
        # training, the large-model layer: forward, then every gradient
        dict(name="qknorm-train-large", op="qknorm_train", dtype=BF16, b=8, l=2048, hq=40, hk=40, d=128, rot=128,
             inter=False, far=0),
        # training on windows of odd sizes in 32 bits that begin somewhere in their documents
        dict(name="qknorm-train-odd", op="qknorm_train", dtype=F32, b=3, l=1021, hq=12, hk=4, d=90, rot=58,
             inter=False, far=100000),
        # serving, one sequence: the next token of the small model's vocabulary
        dict(name="sample-one", op="sample", dtype=BF16, n=1, v=50257, mode="nucleus"),
        # serving, a full batch in which every request has settings of its own
        dict(name="sample-batch", op="sample", dtype=F32, n=256, v=50257, mode="mixed"),
        # serving, a batch over a large vocabulary, the same settings for all
        dict(name="sample-wide", op="sample", dtype=BF16, n=64, v=131072, mode="top"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lattn_step", "lattn_prompt", "lattn_train", "qknorm_fwd", "qknorm_train", "sample"])
    dtype = rng.choice([BF16, BF16, F32])
    case = dict(op=op, dtype=dtype)
    if op.startswith("lattn"):
        dk, dv = rng.choice([(64, 64), (128, 128), (128, 128), (64, 128), (128, 64), (256, 256),
                             (rng.randint(16, 256), rng.randint(16, 256))])
        hk = _log_int(rng, 1, 40)
        group = rng.choice([1, 1, 1, 2, 4])
        h = hk * group
        if op == "lattn_step":
            case.update(b=_log_int(rng, 1, max(2, min(256, 256 * 40 * 128 * 128 // (h * dk * dv)))), l=1)
        else:
            # head elements of the largest listed case of the kind, an eighth of them in 32 bits
            most = 131072 * 16 * 128 if op == "lattn_prompt" else 8 * 2048 * 40 * 128
            rows = max(2, most // (8 if dtype == F32 else 1) * 128 // (h * dk * dv))
            if dk > 128 or dv > 128:
                rows = max(2, rows // 2)
            b = _log_int(rng, 1, max(1, min(16, rows)))
            case.update(b=b, l=_log_int(rng, 1, max(2, min(131072 if op == "lattn_prompt" else 16384, rows // b))))
        case.update(hk=hk, h=h, dk=dk, dv=dv)
        if op == "lattn_train":
            case.update(packed=rng.random() < 0.5)
    elif op.startswith("qknorm"):
        hk = _log_int(rng, 1, 40)
        hq = hk * rng.choice([1, 1, 2, 4])
        d = rng.choice([64, 128, 128, 256, 2 * rng.randint(8, 128)])
        rot = rng.choice([d, d, 2 * rng.randint(1, d // 2)])
        most = 8 * 2048 * 80 * 128 // (1 if op == "qknorm_fwd" else 2)
        rows = max(2, most // (2 if dtype == F32 else 1) // ((hq + hk) * d))
        b = _log_int(rng, 1, max(1, min(16, rows)))
        case.update(b=b, l=_log_int(rng, 1, max(2, min(131072, rows // b))), hq=hq, hk=hk, d=d, rot=rot,
                    inter=rng.random() < 0.3, far=rng.choice([0, 1000, 100000, 1000000]))
    else:
        v = _log_int(rng, 1000, 131072)
        case.update(n=_log_int(rng, 1, max(2, min(256, 256 * 50257 // v))), v=v,
                    mode=rng.choice(["nucleus", "mixed", "top", "floor"]))
    return case


# ---------------------------------------------------------------------------------- the inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = torch.bfloat16 if case["dtype"] == BF16 else torch.float32

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    op = case["op"]
    s = {"op": op, "dt": dt}
    if op.startswith("lattn"):
        b, l, hk, h, dk, dv = (case[n] for n in ("b", "l", "hk", "h", "dk", "dv"))
        # the heads' memories last from 32 to 4096 tokens, evenly in their logarithm
        span = torch.arange(h, device="cuda", dtype=torch.float64) / max(1, h - 1)
        s["log_decay"] = torch.log1p(-torch.exp2(-5.0 - 7.0 * span)).float()
        if op == "lattn_step":
            s.update(q=normal(b, hk, dk), k=normal(b, hk, dk), v=normal(b, h, dv),
                     h=normal(b, h, dk, dv, std=4.0, dtype=torch.float32))
            return s
        s.update(h0=None, reset=None, dh_last=None)
        if op == "lattn_prompt":
            # one projection's output holds the three operands side by side, read in place
            qkv = normal(b, l, 2 * hk * dk + h * dv)
            s.update(q=qkv[..., :hk * dk].unflatten(-1, (hk, dk)),
                     k=qkv[..., hk * dk:2 * hk * dk].unflatten(-1, (hk, dk)),
                     v=qkv[..., 2 * hk * dk:].unflatten(-1, (h, dv)))
            return s
        s.update(q=normal(b, l, hk, dk), k=normal(b, l, hk, dk), v=normal(b, l, h, dv), do=normal(b, l, h, dv))
        if case["packed"]:
            # documents of some 250 tokens one after another; the first goes on from the last window's state
            s["reset"] = uniform(b, l) < 1.0 / 250
            s["h0"] = normal(b, h, dk, dv, std=4.0, dtype=torch.float32)
            s["dh_last"] = normal(b, h, dk, dv, std=0.1, dtype=torch.float32)
        return s
    if op.startswith("qknorm"):
        b, l, hq, hk, d, rot = (case[n] for n in ("b", "l", "hq", "hk", "d", "rot"))
        # the projection's output, read in place
        qk = normal(b, l, (hq + hk) * d, std=1.5)
        s.update(q=qk[..., :hq * d].unflatten(-1, (hq, d)), k=qk[..., hq * d:].unflatten(-1, (hk, d)),
                 w_q=1.0 + normal(d, std=0.1, dtype=torch.float32), w_k=1.0 + normal(d, std=0.1, dtype=torch.float32),
                 inter=case["inter"])
        s["inv_freq"] = torch.pow(ROPE_BASE, -torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot).float()
        start = (uniform(b, 1) * case["far"]).long()
        s["pos"] = start + torch.arange(l, device="cuda")
        if op == "qknorm_train":
            s.update(dqo=normal(b, l, hq, d), dko=normal(b, l, hk, d))
        return s
    n, v = case["n"], case["v"]
    # a language model's logits: most of the vocabulary far below the few tokens that fit
    logits = torch.randn((n, v), generator=gen, device="cuda") * 2.5
    fit = torch.randint(0, v, (n, 40), generator=gen, device="cuda")
    logits.scatter_add_(1, fit, uniform(n, 40) * 10.0)
    s.update(logits=logits.to(dt), u=uniform(n), temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    if case["mode"] == "nucleus":
        s.update(temperature=0.8, top_p=0.95)
    elif case["mode"] == "top":
        s.update(temperature=0.7, top_k=50, top_p=0.9)
    elif case["mode"] == "floor":
        s.update(temperature=1.3, min_p=0.05)
    else:
        # every fourth request is greedy; the others limit the choice in one way or several, or not at all
        kind = torch.randint(0, 4, (n,), generator=gen, device="cuda")
        s["temperature"] = torch.where(kind == 0, 0.0, 0.5 + uniform(n))
        s["top_k"] = torch.where(uniform(n) < 0.5, torch.randint(1, 200, (n,), generator=gen, device="cuda"), 0).int()
        s["top_p"] = torch.where(uniform(n) < 0.6, 0.5 + 0.5 * uniform(n), 1.0)
        s["min_p"] = torch.where(uniform(n) < 0.3, 0.1 * uniform(n), 0.0)
    return s


# ---------------------------------------------------------------------------------- one pass

def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _run_own(s):
    import selective_state_space_85_amd as ss

    op = s["op"]
    if op == "lattn_step":
        return {"o": ss.lattn_step(s["h"], s["q"], s["k"], s["v"], s["log_decay"]), "h": s["h"]}
    if op == "lattn_prompt":
        o, h_last = ss.lattn_fwd(s["q"], s["k"], s["v"], s["log_decay"], return_last_state=True)
        return {"o": o, "h_last": h_last}
    if op == "lattn_train":
        o, h_last = ss.lattn_fwd(s["q"], s["k"], s["v"], s["log_decay"], h0=s["h0"], reset=s["reset"],
                                 return_last_state=True)
        g = ss.lattn_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["do"], h0=s["h0"], reset=s["reset"],
                         dh_last=s["dh_last"], want_dh0=True)
        return {"o": o, "h_last": h_last, **g}
    if op == "qknorm_fwd":
        qo, ko = ss.qknorm_fwd(s["q"], s["k"], s["w_q"], s["w_k"], s["pos"], s["inv_freq"], eps=EPS,
                               interleaved=s["inter"])
        return {"qo": qo, "ko": ko}
    if op == "qknorm_train":
        qo, ko = ss.qknorm_fwd(s["q"], s["k"], s["w_q"], s["w_k"], s["pos"], s["inv_freq"], eps=EPS,
                               interleaved=s["inter"])
        g = ss.qknorm_bwd(s["q"], s["k"], s["w_q"], s["w_k"], s["pos"], s["inv_freq"], s["dqo"], s["dko"], eps=EPS,
                          interleaved=s["inter"])
        return {"qo": qo, "ko": ko, **g}
    return {"token": ss.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                               min_p=s["min_p"])}


def _grouped(x, h):
    """(B, L, heads, D) as (B, h, L, D) in 32 bits, shared heads repeated."""
    return x.float().transpose(1, 2).repeat_interleave(h // x.shape[2], 1)


def _plain_step(s):
    h, g = s["h"], s["h"].shape[1] // s["q"].shape[1]
    q, k = (s[n].float().repeat_interleave(g, 1) for n in ("q", "k"))
    new = torch.exp(s["log_decay"])[:, None, None] * h + k[..., None] * s["v"].float()[..., None, :]
    h.copy_(new)
    o = (q[..., None] * new).sum(2) * q.shape[-1] ** -0.5
    return {"o": o.to(s["dt"]), "h": h}


class _Chunks:
    """The sequence cut into chunks of c rows (the last one filled up with zeros) and the decays
    between rows and chunks: row t takes exp((t - s) log_decay) of row s where no reset lies in (s, t]."""

    def __init__(self, s):
        self.b, self.l = s["q"].shape[:2]
        self.h = s["v"].shape[2]
        c = self.c = min(256, 1 << (self.l - 1).bit_length())
        n = self.n = -(-self.l // c)
        dev = s["q"].device
        g = s["log_decay"].double()
        reset = torch.zeros((self.b, self.l), dtype=torch.bool, device=dev) if s["reset"] is None else s["reset"]
        # the document that each row belongs to; the state h0 belongs to document 0
        doc = torch.nn.functional.pad(reset, (0, n * c - self.l)).long().cumsum(1).view(self.b, 1, n, c)
        last = doc[..., -1]
        before = torch.cat((torch.zeros_like(last[..., :1]), last[..., :-1]), 2)
        i = torch.arange(c, device=dev)
        gap = (i[:, None] - i).clamp(min=0)
        self.pair = (torch.exp(g[:, None, None] * gap).float()[None, :, None]
                     * ((i[:, None] >= i) & (doc[..., :, None] == doc[..., None, :])))  # (b, h, n, t, s)
        # from the state before a chunk to its rows, and from its rows to the state behind it
        self.enter = torch.exp(g[:, None] * (i + 1)).float()[None, :, None] * (doc == before[..., None])
        # rows behind the end hold nothing and put the state off by their count: it is read before them
        tail = torch.zeros((n, 1), dtype=torch.long, device=dev)
        tail[-1] = n * c - self.l
        gap = c - 1 - i - tail
        self.leave = torch.exp(g[:, None, None] * gap.clamp(min=0)).float()[None] * ((doc == last[..., None]) & (gap >= 0))
        # from what chunk j leaves to the state before chunk i, and to the one behind the last (i = n)
        j = torch.arange(n, device=dev)
        to = torch.arange(n + 1, device=dev)[:, None]
        gap = (to - 1 - j) * c - torch.where((to == n) & (j < n - 1), n * c - self.l, 0)
        seen = torch.cat((before, last[..., -1:]), 2)
        self.join = (torch.exp(g[:, None, None] * gap.clamp(min=0)).float()[None]
                     * ((gap >= 0) & (seen[..., :, None] == last[..., None, :])))  # (b, h, i, j)
        rows = (torch.arange(n + 1, device=dev) * c).clamp(max=self.l)
        self.first = torch.exp(g[:, None] * rows).float()[None] * (seen == 0)  # from h0 to the state before chunk i

    def cut(self, x):
        x = torch.nn.functional.pad(_grouped(x, self.h), (0, 0, 0, self.n * self.c - self.l))
        return x.reshape(self.b, self.h, self.n, self.c, -1)

    def whole(self, x):
        """(b, h, n, c, D) back to (B, L, h, D)."""
        return x.flatten(2, 3)[:, :, :self.l].transpose(1, 2)

    def states(self, k, v, h0):
        """The state before every chunk, and behind the last."""
        u = (k * self.leave[..., None]).transpose(-1, -2).contiguous() @ v
        st = (self.join @ u.flatten(3)).unflatten(3, u.shape[3:])
        return st if h0 is None else st + self.first[..., None, None] * h0[:, :, None]

    def adjoints(self, q, do, dh_last):
        """The gradient of the state behind every chunk by what the rows and states after it give, and h0's."""
        w = (q * self.enter[..., None]).transpose(-1, -2).contiguous() @ do
        g = (self.join[..., :-1, :].transpose(-1, -2).contiguous() @ w.flatten(3)).unflatten(3, w.shape[3:])
        first = (self.first[..., :-1, None, None] * w).sum(2)
        if dh_last is not None:
            g = g + self.join[..., -1, :, None, None] * dh_last[:, :, None]
            first = first + self.first[..., -1, None, None] * dh_last
        return g, first


def _plain_attention(s):
    at = _Chunks(s)
    q, k, v = at.cut(s["q"]), at.cut(s["k"]), at.cut(s["v"])
    scale = q.shape[-1] ** -0.5
    p = (q @ k.transpose(-1, -2).contiguous()) * at.pair
    st = at.states(k, v, s["h0"])
    o = p @ v + at.enter[..., None] * (q @ st[:, :, :-1])
    out = {"o": (at.whole(o) * scale).to(s["dt"]), "h_last": st[:, :, -1].contiguous()}
    if s["op"] == "lattn_prompt":
        return out
    do = at.cut(s["do"]) * scale
    ds, dh0 = at.adjoints(q, do, s["dh_last"])
    dp = (do @ v.transpose(-1, -2).contiguous()) * at.pair
    before = st[:, :, :-1].transpose(-1, -2).contiguous()
    dq = dp @ k + at.enter[..., None] * (do @ before)
    dk = dp.transpose(-1, -2).contiguous() @ q + at.leave[..., None] * (v @ ds.transpose(-1, -2).contiguous())
    dv = p.transpose(-1, -2).contiguous() @ do + at.leave[..., None] * (k @ ds)
    hk = s["q"].shape[2]
    for name, g in (("dq", dq), ("dk", dk)):  # shared heads: the sum over those that share them
        out[name] = at.whole(g).unflatten(2, (hk, -1)).sum(3).to(s["dt"])
    out.update(dv=at.whole(dv).to(s["dt"]), dh0=dh0)
    return out


def _rotation(s):
    """cos and sin of pos * inv_freq, the product and its revolutions in 64 bits: (B, L, 1, rot / 2)."""
    turns = s["pos"].double()[..., None] * s["inv_freq"].double() / (2.0 * math.pi)
    angle = ((turns - torch.floor(turns)) * (2.0 * math.pi)).float()[..., None, :]
    return torch.cos(angle), torch.sin(angle)


def _rotate(x, cos, sin, inter):
    n = cos.shape[-1]
    if inter:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., 2 * n:]), -1)


def _plain_qknorm(s):
    cos, sin = _rotation(s)
    out = {}
    for n in ("q", "k"):
        x, w = s[n].float(), s["w_" + n]
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        xr = x * r
        out[n + "o"] = _rotate(xr * w, cos, sin, s["inter"]).to(s["dt"])
        if s["op"] == "qknorm_train":
            g = _rotate(s["d" + n + "o"].float(), cos, -sin, s["inter"])  # turned back
            gw = g * w
            out["d" + n] = (r * (gw - xr * (gw * xr).mean(-1, keepdim=True))).to(s["dt"])
            out["dw_" + n] = (g * xr).sum((0, 1, 2))
    return out


def _column(x, n):
    return x[:, None] if isinstance(x, torch.Tensor) else torch.full((n, 1), x, device="cuda")


def _plain_sample(s):
    n, v = s["logits"].shape
    logits, index = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)
    temperature = _column(s["temperature"], n).double()
    top_k, top_p, min_p = _column(s["top_k"], n), _column(s["top_p"], n).float(), _column(s["min_p"], n).float()
    x = logits.double()
    x = (x - x[:, :1]) / torch.where(temperature > 0, temperature, 1.0)
    w = torch.exp(x)
    place = torch.arange(v, device="cuda")
    w = torch.where((temperature > 0) | (place == 0), w, 0.0)  # greedy: the largest logit, the first of its equals
    w = torch.where((top_k <= 0) | (place < top_k), w, 0.0)
    below = torch.cumsum(w, 1)
    w = torch.where((top_p >= 1) | (below - w < top_p.double() * below[:, -1:]) | (place == 0), w, 0.0)
    w = torch.where((w >= min_p.double()) | (place == 0), w, 0.0)
    below = torch.cumsum(w, 1)
    last = (w > 0).sum(1) - 1
    at = torch.minimum((below <= s["u"].double()[:, None] * below[:, -1:]).sum(1), last)
    return {"token": index.gather(1, at[:, None])[:, 0]}


_PLAIN = {"lattn_step": _plain_step, "lattn_prompt": _plain_attention, "lattn_train": _plain_attention,
          "qknorm_fwd": _plain_qknorm, "qknorm_train": _plain_qknorm, "sample": _plain_sample}


# ---------------------------------------------------------------------------------- the work

def work(case):
    es = 2 if case["dtype"] == BF16 else 4
    op = case["op"]
    if op.startswith("lattn"):
        rows, h, cells = case["b"] * case["l"], case["h"], case["dk"] * case["dv"]
        qk, v = 2 * rows * case["hk"] * case["dk"] * es, rows * h * case["dv"] * es
        state = case["b"] * h * cells * 4
        # a token's head: the state decayed, one outer product added, one product with the query
        if op == "lattn_step":
            return {"bytes": qk + 2 * v + 2 * state + 4 * h, "flops": 5 * rows * h * cells}
        if op == "lattn_prompt":
            return {"bytes": qk + 2 * v + state + 4 * h, "flops": 4 * rows * h * cells}
        extra = rows + 3 * state if case["packed"] else state
        return {"bytes": 2 * qk + 4 * v + state + extra + 4 * h, "flops": 14 * rows * h * cells}
    if op.startswith("qknorm"):
        rows = case["b"] * case["l"]
        n = rows * (case["hq"] + case["hk"]) * case["d"]
        small = 8 * rows + 8 * case["d"] + 2 * case["rot"]
        if op == "qknorm_fwd":
            return {"bytes": 2 * n * es + small, "flops": 7 * n}
        return {"bytes": 4 * n * es + small + 8 * case["d"], "flops": 20 * n}
    # the largest, a difference, a quotient, an exponential, its sum and comparisons
    n = case["n"] * case["v"]
    return {"bytes": n * es + case["n"] * 12, "flops": 8 * n}


# ---------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    if case["op"] == "lattn_train" and case["l"] > 20000:
        return None
    s = prepare(case, seed)
    if case["op"].startswith("lattn"):
        return _exact_attention(s)
    return _exact_qknorm(s) if case["op"].startswith("qknorm") else _exact_sample(s)


def _exact_attention(s):
    # token by token, as the recurrence is written
    h = s["v"].shape[-2]
    a = s["log_decay"].double().exp()[:, None, None]
    hk, dk = s["q"].shape[-2:]
    scale = 1.0 / math.sqrt(dk)
    head = torch.arange(h, device="cuda") // (h // hk)
    if s["op"] == "lattn_step":
        q, k = s["q"].double()[:, head], s["k"].double()[:, head]
        st = s["h"].double() * a + torch.einsum("bhi,bhj->bhij", k, s["v"].double())
        return {"o": torch.einsum("bhi,bhij->bhj", q, st) * scale, "h": st}
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    nb, nl = q.shape[:2]
    st = torch.zeros((nb, h, dk, v.shape[-1]), dtype=torch.float64, device="cuda") if s["h0"] is None else s["h0"].double()
    reset = s["reset"]
    train = s["op"] == "lattn_train"
    o = torch.empty_like(v)
    if train:
        do = s["do"].double() * scale
        dq, dk_, dv = (torch.empty((nb, nl, h, w), dtype=torch.float64, device="cuda") for w in (dk, dk, v.shape[-1]))
    shared = h == hk
    for t in range(nl):
        kt, qt = (k[:, t], q[:, t]) if shared else (k[:, t, head], q[:, t, head])
        st = st * a
        if reset is not None:
            st = st * (~reset[:, t, None, None, None])
        st.addcmul_(kt[..., None], v[:, t, :, None, :])
        o[:, t] = (qt[..., None, :] @ st)[..., 0, :]
        if train:
            dq[:, t] = (st @ do[:, t, ..., None])[..., 0]
    out = {"o": o * scale, "h_last": st.clone()}
    if not train:
        return out
    g = torch.zeros_like(st) if s["dh_last"] is None else s["dh_last"].double()
    for t in range(nl - 1, -1, -1):
        kt, qt = (k[:, t], q[:, t]) if shared else (k[:, t, head], q[:, t, head])
        g = torch.addcmul(g, qt[..., None], do[:, t, :, None, :])
        dv[:, t] = (kt[..., None, :] @ g)[..., 0, :]
        dk_[:, t] = (g @ v[:, t, ..., None])[..., 0]
        g = g * a
        if reset is not None:
            g = g * (~reset[:, t, None, None, None])
    per = h // hk
    out.update(dq=dq.view(nb, nl, hk, per, dk).sum(3), dk=dk_.view(nb, nl, hk, per, dk).sum(3), dv=dv, dh0=g)
    return out


def _exact_qknorm(s):
    # pairs as complex numbers; the gradients by automatic differentiation
    rot = 2 * s["inv_freq"].shape[0]
    angle = s["pos"].double()[..., None, None] * s["inv_freq"].double()
    turn = torch.complex(angle.cos(), angle.sin())
    out = {}
    for n in ("q", "k"):
        x, w = s[n].double().requires_grad_(), s["w_" + n].double().requires_grad_()
        y = w * x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
        if s["inter"]:
            z = torch.view_as_complex(y[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous()) * turn
            turned = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * turn
            turned = torch.cat((z.real, z.imag), -1)
        y = torch.cat((turned, y[..., rot:]), -1)
        out[n + "o"] = y.detach()
        if s["op"] == "qknorm_train":
            out["d" + n], out["dw_" + n] = torch.autograd.grad(y, (x, w), s["d" + n + "o"].double())
    return out


def _exact_sample(s):
    # row by row on the host
    logits = s["logits"].float().cpu().numpy().astype(np.float64)
    n, v = logits.shape
    rows = {name: np.broadcast_to(s[name].cpu().numpy() if isinstance(s[name], torch.Tensor) else np.float32(s[name]), (n,))
            for name in ("temperature", "top_k", "top_p", "min_p", "u")}
    tokens = []
    for i in range(n):
        order = np.argsort(-logits[i], kind="stable")
        t, k, p, m, u = (float(rows[name][i]) for name in ("temperature", "top_k", "top_p", "min_p", "u"))
        if t <= 0:
            tokens.append(int(order[0]))
            continue
        if k > 0:
            order = order[:int(k)]
        w = np.exp((logits[i][order] - logits[i][order[0]]) / t)
        if p < 1:
            below = np.concatenate(([0.0], np.cumsum(w)[:-1]))
            keep = max(1, int((below < p * w.sum()).sum()))
            order, w = order[:keep], w[:keep]
        keep = max(1, int((w >= m).sum()))
        order, w = order[:keep], w[:keep]
        at = int(np.searchsorted(np.cumsum(w), u * w.sum(), side="right"))
        tokens.append(int(order[min(at, int((w > 0).sum()) - 1)]))
    return {"token": torch.tensor(tokens, device="cuda")}
