"""Linear attention, its norms and sampling as a model uses them: one after another, in graphs, on
streams of their own, on long rows, and in the example."""
import os
import sys

import numpy as np
import pytest
import torch

import attn_ref as ref
from gpu_util import host64, say

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ss():
    import selective_state_space_85_amd as ss

    assert torch.cuda.is_available()
    return ss


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import recurrent_lm
    finally:
        sys.path.pop(0)
    return recurrent_lm


def layer(dtype, b, l, h, d, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, dtype=dtype):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)

    qkv = normal(b, l, 3 * h * d)
    small = dict(w_q=1 + 0.1 * normal(d, dtype=F32), w_k=1 + 0.1 * normal(d, dtype=F32),
                 pos=torch.arange(l, device="cuda").expand(b, l).contiguous(),
                 inv_freq=torch.tensor(10000.0 ** (-np.arange(d // 2) / (d // 2)), dtype=F32, device="cuda"),
                 log_decay=torch.tensor(np.log1p(-np.exp2(-4.0 - np.arange(h))), dtype=F32, device="cuda"))
    return qkv, small, normal


def run_layer(ss, qkv, small, h, workspace=None, **more):
    q, k, v = (t.unflatten(-1, (h, -1)) for t in qkv.chunk(3, -1))
    qn, kn = ss.qknorm_fwd(q, k, small["w_q"], small["w_k"], small["pos"], small["inv_freq"])
    return ss.lattn_fwd(qn, kn, v, small["log_decay"], workspace=workspace, **more), (q, k, v, qn, kn)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_then_tokens(ss, dtype):
    """A prompt through norms and attention, then token by token, then a token sampled from what comes
    out, against 64 bits."""
    say("together", dtype)
    b, l, h, d, cut = 2, 90, 3, 32, 70
    qkv, small, _ = layer(dtype, b, l, h, d, 1)
    part = dict(small, pos=small["pos"][:, :cut].contiguous())
    (o, state), _ = run_layer(ss, qkv[:, :cut].contiguous(), part, h, return_last_state=True)
    rows = [o]
    for t in range(cut, l):
        q, k, v = (x.unflatten(-1, (h, d)) for x in qkv[:, t].chunk(3, -1))
        q, k = ss.qknorm_fwd(q, k, small["w_q"], small["w_k"], small["pos"][:, t].contiguous(), small["inv_freq"])
        rows.append(ss.lattn_step(state, q, k, v, small["log_decay"])[:, None])
    got = host64(torch.cat(rows, 1))
    x = host64(qkv).reshape(b, l, 3, h, d)
    pos, inv = small["pos"].cpu().numpy(), host64(small["inv_freq"])
    q = ref.qknorm(x[:, :, 0], host64(small["w_q"]), pos, inv, 1e-6, False)
    k = ref.qknorm(x[:, :, 1], host64(small["w_k"]), pos, inv, 1e-6, False)
    want, _ = ref.lattn(q, k, x[:, :, 2], host64(small["log_decay"]), d ** -0.5)
    # bf16: o, q and k are rounded, and the state or q k^T, half a step (2^-8) each; fp32: the norms' 2^-20 and
    # the sums'
    tol = 4 * 2.0 ** -8 if dtype is BF16 else 2 * 2.0 ** -20 + 4 * 2.0 ** -24 * np.sqrt(d + l)
    assert np.linalg.norm(got - want) <= tol * np.linalg.norm(want)
    logits = torch.cat(rows, 1).flatten(2).reshape(b * l, h * d).contiguous()
    u = torch.rand((b * l,), device="cuda")
    token = ss.sample(logits, u, temperature=0.5, top_k=20, top_p=0.9)
    l64, u64 = host64(logits), host64(u)
    assert token.tolist() == [ref.sample_row(l64[i], u64[i], 0.5, 20, float(np.float32(0.9))) for i in range(b * l)]


def test_in_graphs(ss):
    """Forward, backward, one token and sampling, captured and replayed with other inputs, with eager work
    between the replays."""
    say("attention in graphs")
    b, l, h, d, vocab = 1, 1100, 2, 64, 1000  # cut in segments: the workspace holds their states
    qkv, small, normal = layer(BF16, b, l, h, d, 2)
    do, h0 = normal(b, l, h, d), normal(b, h, d, d, dtype=F32)
    logits, u = normal(7, vocab), torch.rand((7,), device="cuda")
    token_qkv = normal(b, 3 * h * d)
    reset = torch.zeros((b, l), dtype=torch.bool, device="cuda")
    ws = torch.empty(max(1, ss.lattn_workspace_bytes(b, l, h, h, d, d, BF16),
                         ss.lattn_bwd_workspace_bytes(b, l, h, h, d, d, BF16)), dtype=torch.uint8, device="cuda")
    norm_ws = torch.empty(ss.qknorm_bwd_workspace_bytes(b * l, h, h, d), dtype=torch.uint8, device="cuda")
    state = torch.zeros((b, h, d, d), device="cuda")

    def step():
        state.zero_()
        (o, last), (q, k, v, qn, kn) = run_layer(ss, qkv, small, h, ws, h0=h0, reset=reset, return_last_state=True)
        g = ss.lattn_bwd(qn, kn, v, small["log_decay"], do, h0=h0, reset=reset, want_dh0=True, workspace=ws)
        n = ss.qknorm_bwd(q, k, small["w_q"], small["w_k"], small["pos"], small["inv_freq"], g["dq"], g["dk"],
                          workspace=norm_ws)
        tq, tk, tv = (t.unflatten(-1, (h, d)) for t in token_qkv.chunk(3, -1))
        t = ss.lattn_step(state, tq, tk, tv, small["log_decay"])
        pick = ss.sample(logits, u, temperature=0.7, top_k=50, top_p=0.9, min_p=0.01)
        return [o, last, t, pick, state] + [g[x] for x in sorted(g)] + [n[x] for x in sorted(n)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(3, 7):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        for x in (qkv, do, h0, logits, token_qkv):
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        u.copy_(torch.rand(u.shape, generator=gen, device="cuda"))
        reset.copy_(torch.rand(reset.shape, generator=gen, device="cuda") < 0.01 * (seed - 3))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)), seed


def test_on_other_streams(ss):
    """The calls run on the current stream, two of them beside each other with workspaces of their own."""
    say("attention on streams")
    b, l, h, d = 1, 2200, 4, 128
    made = [layer(BF16, b, l, h, d, s) for s in (8, 9)]
    want = [run_layer(ss, x, small, h)[0] for x, small, _ in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    spaces = [torch.empty(ss.lattn_workspace_bytes(b, l, h, h, d, d, BF16), dtype=torch.uint8, device="cuda") for _ in made]
    assert spaces[0].numel() > 0
    for _ in range(3):
        got = []
        for st, (x, small, _), ws in zip(streams, made, spaces):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(run_layer(ss, x, small, h, ws)[0])
        for st in streams:
            torch.cuda.current_stream().wait_stream(st)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_offsets_beyond_32_bits(ss):
    """Operands that span more than 2^32 bytes, read in place and written whole."""
    say("attention beyond 32 bits")
    l, wide = 150000, 16384  # 4.9 GB of bfloat16
    big = torch.empty((1, l, wide), dtype=BF16, device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(10)
    part = torch.randn((1, l, 3 * 64), generator=gen, device="cuda").to(BF16)
    at = wide - 3 * 64
    big[..., at:] = part
    small = layer(BF16, 1, l, 1, 64, 11)[1]
    want, _ = run_layer(ss, part, small, 1)
    got, _ = run_layer(ss, big[..., at:], small, 1)
    assert torch.equal(got, want)
    say("   backward")
    q, k, v = (t.unflatten(-1, (1, 64)) for t in big[..., at:].chunk(3, -1))
    q2, k2, v2 = (t.unflatten(-1, (1, 64)) for t in part.chunk(3, -1))
    g, w = ss.lattn_bwd(q, k, v, small["log_decay"], v), ss.lattn_bwd(q2, k2, v2, small["log_decay"], v2)
    assert all(torch.equal(g[n], w[n]) for n in g)
    del big, q, k, v
    say("   sample")
    rows, vocab = 40000, 65536  # 5.2 GB
    logits = torch.empty((rows, vocab), dtype=BF16, device="cuda")
    logits[:] = torch.randn((vocab,), generator=gen, device="cuda").to(BF16)
    logits[-3:] = torch.randn((3, vocab), generator=gen, device="cuda").to(BF16)
    u = torch.rand((rows,), generator=gen, device="cuda")
    token = ss.sample(logits, u, top_p=0.9)
    assert torch.equal(token[-3:], ss.sample(logits[-3:].clone(), u[-3:].contiguous(), top_p=0.9))
    assert torch.equal(token[:2], ss.sample(logits[:2].clone(), u[:2].contiguous(), top_p=0.9))


def test_example_gradients(ss, example):
    """The example's attention layer against automatic differentiation of the same in 64 bits."""
    say("example: gradients")
    b, l, h, d = 2, 40, 2, 16
    gen = torch.Generator().manual_seed(12)
    leaf = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64).float().double().requires_grad_()  # noqa: E731
    qkv, w_q, w_k = leaf(b, l, 3 * h * d), leaf(d), leaf(d)
    do = torch.randn(b, l, h * d, generator=gen, dtype=torch.float64).float().double()
    reset = torch.rand(b, l, generator=gen) < 0.1
    log_decay = torch.tensor([-0.1, -0.01], dtype=torch.float64).float().double()
    inv = torch.tensor(10000.0 ** (-np.arange(4) / 4)).float().double()
    at = torch.arange(l)
    pos = at - torch.where(reset, at, 0).cummax(1).values
    doc = reset.long().cumsum(1)

    def norm(x, w):
        y = w * x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        ang = pos[..., None, None] * inv
        y1, y2 = y[..., :4], y[..., 4:8]
        return torch.cat((y1 * ang.cos() - y2 * ang.sin(), y2 * ang.cos() + y1 * ang.sin(), y[..., 8:]), -1)

    q, k, v = (t.unflatten(-1, (h, d)) for t in qkv.chunk(3, -1))
    scores = torch.einsum("bthd,bshd->bhts", norm(q, w_q), norm(k, w_k))
    gap = (at[:, None] - at).clamp(min=0)
    mask = (at[:, None] >= at) & (doc[:, :, None] == doc[:, None, :])
    weights = torch.exp(log_decay[:, None, None] * gap) * mask[:, None]
    o = torch.einsum("bhts,bshd->bthd", scores * weights, v).flatten(2) * d ** -0.5
    o.backward(do)
    dev = [t.detach().float().cuda().requires_grad_() for t in (qkv, w_q, w_k)]
    got = example.LinearAttention.apply(*dev, example.positions(reset.cuda()), inv.float().cuda(),
                                        log_decay.float().cuda(), reset.cuda())
    got.backward(do.float().cuda())
    for name, x, y in (("o", got, o), *((n, t.grad, w.grad) for n, t, w in zip(("dqkv", "dw_q", "dw_k"), dev, (qkv, w_q, w_k)))):
        e = float((x.detach().cpu().double() - y.detach()).norm() / y.detach().norm())
        # the norms' roundings both ways (2^-20 each) and sums of up to L + d terms
        assert e <= 4 * 2.0 ** -20 + 4 * 2.0 ** -24 * (l + d) ** 0.5, (name, e)


def test_example_runs(ss, example):
    say("example: training with attention")
    model, history = example.train(steps=4, batch=4, length=97, vocab=61, dim=128, hidden=192, layers=2, mix="attention",
                                   report=lambda s: print(s, flush=True))
    assert all(np.isfinite(history))
    # bf16 activations through a few roundings each way: 2^-8 each, of the largest logit
    assert example.states_agree(model, 61, length=70) < 0.05
    prompt = torch.randint(0, 61, (3, 5), device="cuda")
    tokens = example.generate(model, prompt, 6, temperature=0.8, top_k=20, top_p=0.95)
    assert tokens.shape == (3, 6) and int(tokens.min()) >= 0 and int(tokens.max()) < 61
    again = example.generate(model, prompt, 6, temperature=0.8, top_k=20, top_p=0.95)
    assert torch.equal(tokens, again)
