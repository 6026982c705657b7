#!/usr/bin/env python3
"""A small recurrent language model trained on one MI355X with the library's operators.

    python examples/recurrent_lm.py [--steps 60] [--layers 2] [--dim 256] [--mix attention] ...

Each layer mixes along the sequence and then across channels:

    x += W_out glr(conv1d_silu(W_in x), gates W_r x, W_i x)     (conv1d_silu, glr_fwd / glr_bwd)
    x += W_down glu(x)                                           (glu_fwd / glu_bwd)

or, with --mix attention, along the sequence by linear attention with a decay for each head:

    q, k, v = W_in x;  x += W_out lattn(qknorm(q, k), v)         (qknorm_fwd / _bwd, lattn_fwd / lattn_bwd)

after a normalisation each, and the loss is the cross entropy of the vocabulary projection
(xent_fwd / xent_bwd).  Plain projections, the normalisation and the optimiser are torch's.  The
text is synthetic: every token repeats the one `lag` places before it with probability 0.9,
documents of random length follow one another in each row, and the recurrence is reset where
one starts.  After training the same weights run token by token from the recurrence's state
(glr_step, lattn_step), which is checked against the parallel form, and continue a prompt with
sampled tokens (sample).
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import selective_state_space_85_amd as ss  # noqa: E402


class Recurrence(torch.autograd.Function):
    """glr_fwd with the states kept for glr_bwd; x, r and i are slices of one tensor."""

    @staticmethod
    def forward(ctx, xri, decay, reset):
        b, l, d3 = xri.shape
        d = d3 // 3
        x, r, i = xri[..., :d], xri[..., d:2 * d], xri[..., 2 * d:]
        ckpt = torch.empty(ss.glr_ckpt_shape(b, l, d), device=xri.device)
        y = ss.glr_fwd(x, r, i, decay, reset=reset, ckpt=ckpt)
        ctx.save_for_backward(xri, decay, reset, ckpt)
        return y

    @staticmethod
    def backward(ctx, dy):
        xri, decay, reset, ckpt = ctx.saved_tensors
        d = xri.shape[-1] // 3
        out = torch.empty_like(xri)
        g = ss.glr_bwd(xri[..., :d], xri[..., d:2 * d], xri[..., 2 * d:], decay, dy.contiguous(), reset=reset,
                       ckpt=ckpt, want_dh0=False, out=out)
        return out, g["ddecay"], None


class LinearAttention(torch.autograd.Function):
    """qknorm_fwd and lattn_fwd on the slices of one projection's output, and their gradients; the heads'
    queries and keys are formed again in the backward."""

    @staticmethod
    def forward(ctx, qkv, w_q, w_k, pos, inv_freq, log_decay, reset):
        q, k, v = LinearAttention.slices(qkv, log_decay.shape[0])
        qn, kn = ss.qknorm_fwd(q, k, w_q, w_k, pos, inv_freq)
        ctx.save_for_backward(qkv, w_q, w_k, pos, inv_freq, log_decay, reset)
        return ss.lattn_fwd(qn, kn, v, log_decay, reset=reset).flatten(2)

    @staticmethod
    def backward(ctx, do):
        qkv, w_q, w_k, pos, inv_freq, log_decay, reset = ctx.saved_tensors
        heads = log_decay.shape[0]
        q, k, v = LinearAttention.slices(qkv, heads)
        qn, kn = ss.qknorm_fwd(q, k, w_q, w_k, pos, inv_freq)
        g = ss.lattn_bwd(qn, kn, v, log_decay, do.contiguous().unflatten(2, (heads, -1)), reset=reset)
        n = ss.qknorm_bwd(q, k, w_q, w_k, pos, inv_freq, g["dq"], g["dk"])
        return torch.cat((n["dq"], n["dk"], g["dv"]), 2).flatten(2), n["dw_q"], n["dw_k"], None, None, None, None

    @staticmethod
    def slices(qkv, heads):
        """q, k and v (..., heads, width) in place."""
        return (t.unflatten(-1, (heads, -1)) for t in qkv.chunk(3, -1))


class GatedProjection(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up):
        ctx.save_for_backward(x, w_gate, w_up)
        return ss.glu_fwd(x, w_gate, w_up)

    @staticmethod
    def backward(ctx, dh):
        g = ss.glu_bwd(*ctx.saved_tensors, dh.contiguous())
        return g["dx"], g["dw_gate"], g["dw_up"]


class VocabularyLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, target):
        loss, lse = ss.xent_fwd(x, w, target)
        ctx.save_for_backward(x, w, target, lse)
        return loss

    @staticmethod
    def backward(ctx, dloss):
        g = ss.xent_bwd(*ctx.saved_tensors, dloss.contiguous())
        return g["dx"], g["dw"], None


class Convolution(torch.autograd.Function):
    """conv1d_silu; its gradient in plain torch (the library has the forward only)."""

    @staticmethod
    def forward(ctx, x, weight, bias):
        ctx.save_for_backward(x, weight, bias)
        return ss.conv1d_silu(x, weight, bias)

    @staticmethod
    def backward(ctx, du):
        x, weight, bias = ctx.saved_tensors
        with torch.enable_grad():
            x, weight, bias = (t.detach().requires_grad_() for t in (x, weight, bias))
            l, width = x.shape[1], weight.shape[1]
            xp = torch.nn.functional.pad(x.float(), (0, 0, width - 1, 0))
            pre = bias + sum(weight[:, k] * xp[:, k:k + l] for k in range(width))
            out = torch.nn.functional.silu(pre)
            return torch.autograd.grad(out, (x, weight, bias), du.float())


def norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


def positions(reset):
    """Each token's place in its document."""
    at = torch.arange(reset.shape[1], device=reset.device)
    return at - torch.where(reset, at, 0).cummax(1).values


class Model:
    HEADS = 4

    def __init__(self, vocab, dim, hidden, layers, gen, mix="glr"):
        def weight(rows, cols):
            return (torch.randn((rows, cols), generator=gen, device="cuda") / cols ** 0.5).requires_grad_()

        # every parameter is held in float32; the matrices are rounded to bfloat16 where they are used
        self.embed = torch.randn((vocab, dim), generator=gen, device="cuda").requires_grad_()
        self.mix = mix
        self.layers = []
        if mix == "attention":
            # memories of 8 to 512 tokens; positions turn half of each head
            width = dim // self.HEADS
            self.log_decay = torch.log1p(-torch.exp2(-3.0 - 6.0 * torch.arange(self.HEADS, device="cuda") / (self.HEADS - 1)))
            self.inv_freq = 10000.0 ** (-torch.arange(0, width // 2, 2, device="cuda") / (width // 2))
        for _ in range(layers if mix == "attention" else 0):
            self.layers.append({
                "in": weight(3 * dim, dim), "out": weight(dim, dim),
                "w_q": torch.ones((width,), device="cuda").requires_grad_(),
                "w_k": torch.ones((width,), device="cuda").requires_grad_(),
                "gate": weight(hidden, dim), "up": weight(hidden, dim), "down": weight(dim, hidden)})
        for _ in range(layers if mix == "glr" else 0):
            k = torch.exp(torch.empty((dim,), device="cuda").uniform_(-7.0, -2.5, generator=gen))
            self.layers.append({
                "in": weight(dim, dim), "gates": weight(2 * dim, dim), "out": weight(dim, dim),
                "conv": (torch.randn((dim, 4), generator=gen, device="cuda") * 0.3).requires_grad_(),
                "conv_bias": torch.zeros((dim,), device="cuda").requires_grad_(),
                "decay": torch.log(torch.expm1(k / 8.0)).requires_grad_(),
                "gate": weight(hidden, dim), "up": weight(hidden, dim), "down": weight(dim, hidden)})
        self.head = weight(vocab, dim)

    def parameters(self):
        return [self.embed, self.head] + [p for layer in self.layers for p in layer.values()]

    def rounded(self):
        """(embedding, head, layers) as the operators take them."""
        matrices = ("in", "gates", "out", "gate", "up", "down")
        return (self.embed.bfloat16(), self.head.bfloat16(),
                [{n: w.bfloat16() if n in matrices else w for n, w in layer.items()} for layer in self.layers])

    def features(self, tokens, reset, weights):
        embed, _, layers = weights
        x = embed[tokens]
        for p in layers:
            n = norm(x)
            if self.mix == "attention":
                mixed = LinearAttention.apply((n @ p["in"].t()).contiguous(), p["w_q"], p["w_k"], positions(reset),
                                              self.inv_freq, self.log_decay, reset)
            else:
                u = Convolution.apply((n @ p["in"].t()).contiguous(), p["conv"], p["conv_bias"])
                mixed = Recurrence.apply(torch.cat((u, n @ p["gates"].t()), -1), p["decay"], reset)
            x = x + mixed @ p["out"].t()
            x = x + GatedProjection.apply(norm(x), p["gate"], p["up"]) @ p["down"].t()
        return norm(x)

    def loss(self, tokens, reset):
        weights = self.rounded()
        x = self.features(tokens[:, :-1], reset[:, :-1].contiguous(), weights)
        target = tokens[:, 1:].masked_fill(reset[:, 1:], -100)  # nothing foretells a document's first token
        loss = VocabularyLoss.apply(x, weights[1], target.contiguous())
        return loss.sum() / (target >= 0).sum()

    @torch.no_grad()
    def start(self, batch):
        d = self.embed.shape[1]
        if self.mix == "attention":
            w = d // self.HEADS
            return [{"h": torch.zeros((batch, self.HEADS, w, w), device="cuda"),
                     "pos": torch.zeros((batch,), dtype=torch.int64, device="cuda")} for _ in self.layers]
        return [{"h": torch.zeros((batch, d), device="cuda"),
                 "window": torch.zeros((batch, 4, d), dtype=torch.bfloat16, device="cuda")} for _ in self.layers]

    @torch.no_grad()
    def step(self, token, state, weights):
        """One token (batch,) past the states; the logits of the next."""
        embed, head, layers = weights
        x = embed[token]
        for p, s in zip(layers, state):
            n = norm(x)
            if self.mix == "attention":
                q, k, v = LinearAttention.slices(n @ p["in"].t(), self.HEADS)
                q, k = ss.qknorm_fwd(q, k, p["w_q"], p["w_k"], s["pos"], self.inv_freq)
                s["pos"] += 1
                x = x + ss.lattn_step(s["h"], q, k, v, self.log_decay).flatten(1) @ p["out"].t()
                x = x + ss.glu_fwd(norm(x), p["gate"], p["up"]) @ p["down"].t()
                continue
            s["window"] = torch.cat((s["window"][:, 1:], (n @ p["in"].t())[:, None]), 1)
            u = ss.conv1d_silu(s["window"], p["conv"], p["conv_bias"])[:, -1].contiguous()
            gates = n @ p["gates"].t()
            d = u.shape[1]
            x = x + ss.glr_step(s["h"], u, gates[:, :d], gates[:, d:], p["decay"]) @ p["out"].t()
            x = x + ss.glu_fwd(norm(x), p["gate"], p["up"]) @ p["down"].t()
        return norm(x) @ head.t()


def text(batch, length, vocab, lag, gen):
    """Tokens that mostly repeat the one `lag` places before, and where documents start."""
    tokens = torch.randint(0, vocab, (batch, length), generator=gen, device="cuda")
    copy = torch.rand((batch, length), generator=gen, device="cuda") < 0.9
    reset = torch.rand((batch, length), generator=gen, device="cuda") < 1.0 / 200
    reset[:, 0] = True
    since = torch.zeros((batch,), dtype=torch.int64, device="cuda")
    for t in range(length):
        since = torch.where(reset[:, t], 0, since + 1)
        if t >= lag:
            tokens[:, t] = torch.where(copy[:, t] & (since >= lag), tokens[:, t - lag], tokens[:, t])
    return tokens, reset


def train(steps=60, batch=16, length=257, vocab=509, dim=256, hidden=704, layers=2, lag=2, lr=5e-3, seed=0,
          mix="glr", report=print):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    model = Model(vocab, dim, hidden, layers, gen, mix)
    opt = torch.optim.Adam(model.parameters(), lr=lr, betas=(0.9, 0.98))
    history = []
    for step in range(steps):
        tokens, reset = text(batch, length, vocab, lag, gen)
        loss = model.loss(tokens, reset)
        opt.zero_grad()
        loss.backward()
        opt.step()
        history.append(float(loss.detach()))
        if step % 10 == 0 or step == steps - 1:
            report("step %3d loss %.3f" % (step, history[-1]))
    return model, history


@torch.no_grad()
def states_agree(model, vocab, length=100, batch=3, seed=1):
    """The largest difference between token-by-token logits and the parallel form's."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    tokens = torch.randint(0, vocab, (batch, length), generator=gen, device="cuda")
    reset = torch.zeros((batch, length), dtype=torch.bool, device="cuda")
    weights = model.rounded()
    want = model.features(tokens, reset, weights) @ weights[1].t()
    state = model.start(batch)
    got = torch.stack([model.step(tokens[:, t].contiguous(), state, weights) for t in range(length)], 1)
    return float((got.float() - want.float()).abs().max() / want.float().abs().max())


@torch.no_grad()
def generate(model, prompt, count, seed=2, **limits):
    """`count` tokens sampled after the prompt (batch, length); limits as of ss.sample."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    weights, state = model.rounded(), model.start(prompt.shape[0])
    for t in range(prompt.shape[1]):
        logits = model.step(prompt[:, t].contiguous(), state, weights)
    tokens = []
    for _ in range(count):
        u = torch.rand((prompt.shape[0],), generator=gen, device="cuda")
        tokens.append(ss.sample(logits, u, **limits))
        logits = model.step(tokens[-1], state, weights)
    return torch.stack(tokens, 1)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("steps", 60), ("batch", 16), ("length", 257), ("vocab", 509), ("dim", 256), ("hidden", 704),
                        ("layers", 2), ("lag", 2)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--mix", choices=("glr", "attention"), default="glr")
    args = ap.parse_args()
    model, _ = train(**vars(args))
    print("token by token against the parallel form: %.1e of the largest logit" % states_agree(model, args.vocab))
    prompt = torch.randint(0, args.vocab, (1, 8), device="cuda")
    print("prompt", prompt[0].tolist(), "continues", generate(model, prompt, 8, temperature=0.7, top_p=0.9)[0].tolist())


if __name__ == "__main__":
    main()
