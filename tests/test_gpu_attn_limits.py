"""Linear attention and its norms on the GPU at sizes whose launches fill much of a grid."""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ss():
    import selective_state_space_85_amd as ss

    assert torch.cuda.is_available()
    return ss


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def test_attention_of_many_sequences(ss):
    """Three million sequences of one row: o = scale (q . k) v, and its gradients."""
    n = 3000011
    say("lattn", n, "sequences")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    q, k, v, do = (normal(gen, n, 1, 1, 4) for _ in range(4))
    decay = torch.tensor([-0.1], device="cuda")
    o, last = ss.lattn_fwd(q, k, v, decay, return_last_state=True)
    g = ss.lattn_bwd(q, k, v, decay, do)
    torch.cuda.synchronize()
    q, k, v, do = (t.double() for t in (q, k, v, do))
    qk, dov = 0.5 * (q * k).sum(-1, keepdim=True), 0.5 * (do * v).sum(-1, keepdim=True)
    # sums of four products, a product by the scale and one by a row: 6 roundings of half a step, 2^-24 each
    for name, got, want in (("o", o, qk * v), ("h_last", last, k[:, 0, :, :, None] * v[:, 0, :, None, :]),
                            ("dq", g["dq"], dov * k), ("dk", g["dk"], dov * q), ("dv", g["dv"], qk * do)):
        say("   %s %.2e" % (name, off(got, want)))
        assert off(got, want) <= 6 * 2.0 ** -24, name
        assert torch.isfinite(got).all()


def test_one_token_of_many_heads(ss):
    n = 4500001
    say("lattn_step", n, "sequences")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    h = normal(gen, n, 1, 2, 3)
    q, k, v = normal(gen, n, 1, 2), normal(gen, n, 1, 2), normal(gen, n, 1, 3)
    decay = torch.tensor([-0.5], device="cuda")
    want_h = h.double() * decay.double().exp() + k.double()[..., None] * v.double()[..., None, :]
    want = (q.double()[..., None] * want_h).sum(2) * 2 ** -0.5
    o = ss.lattn_step(h, q, k, v, decay)
    torch.cuda.synchronize()
    # the decay, two products and a sum; two products, a sum and the scale besides
    assert off(h, want_h) <= 4 * 2.0 ** -24
    assert off(o, want) <= 8 * 2.0 ** -24


def test_norms_of_many_tokens(ss):
    n, w = (1 << 23) + 3, 8
    say("qknorm", n, "tokens")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    q, k, dqo, dko = (normal(gen, n, 1, w) for _ in range(4))
    w_q, w_k = 1 + 0.1 * normal(gen, w), 1 + 0.1 * normal(gen, w)
    pos = torch.randint(0, 100000, (n,), generator=gen, device="cuda")
    inv = torch.tensor([1.0, 0.01], device="cuda")
    out = ss.qknorm_fwd(q, k, w_q, w_k, pos, inv, eps=1e-5)
    g = ss.qknorm_bwd(q, k, w_q, w_k, pos, inv, dqo, dko, eps=1e-5)
    torch.cuda.synchronize()
    angle = pos.double()[:, None, None] * inv.double()
    cos, sin = angle.cos(), angle.sin()

    def turn(y, s):
        a, b = y[..., :2], y[..., 2:4]
        return torch.cat((a * cos - b * s, b * cos + a * s, y[..., 4:]), -1)

    # roundings of the norm and the turn: of x r w 2, of the root 2, of the turn 3, of cosine and sine 2^-23 each
    tol = 7 * 2.0 ** -24 + 2 * 2.0 ** -23
    for name, x, wt, dy, y, i in (("q", q, w_q, dqo, out[0], 0), ("k", k, w_k, dko, out[1], 1)):
        x, wt, dy = x.double(), wt.double(), dy.double()
        r = (x.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
        assert off(y, turn(x * r * wt, sin)) <= tol, name
        back = turn(dy, -sin)
        gw = back * wt
        dx = r * (gw - x * r * (gw * x * r).mean(-1, keepdim=True))
        assert off(g["d" + name], dx) <= 4 * tol, name  # the difference of two such terms
        dw = (back * x * r).sum((0, 1))
        # sums of 2^23 terms of mixed signs, relative to the terms' norm: each term's error, and one rounding for each
        # addition of a running sum, which after i of them is sqrt(i) terms large.  256 in a lane, 32 groups of
        # lanes, 16 and 64 runs of workgroups' sums one after another.
        scale = float((back * x * r).square().sum((0, 1)).sqrt().norm())
        e = float((g["dw_" + name].double() - dw).norm()) / scale
        say("   dw_%s %.2e" % (name, e))
        assert e <= tol + 2.0 ** -24 * (256 + 32 + 16 + 64) ** 0.5, name


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(64, 128), (72, 91), (3, 40), (256, 5)])
def test_one_row_of_long_sequences(ss, dtype, dk, dv):
    """One row each of sequences that lie more than 2^20 elements apart, read in place."""
    say("lattn one row", dtype, dk, dv)
    b, l, hk, h, wide = 3, 40, 2, 4, 32768
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    rows = torch.full((b, l, wide), float("nan"), dtype=dtype, device="cuda")
    rows[:, 17:18] = normal(gen, b, 1, wide).to(dtype)
    row, at, views = rows[:, 17:18], 0, []
    for heads, width in ((hk, dk), (hk, dk), (h, dv), (h, dv)):
        views.append(row[..., at:at + heads * width].unflatten(-1, (heads, width)))
        at += (heads * width + 7) // 8 * 8  # the same alignment as by themselves
    decay = -torch.rand((h,), generator=gen, device="cuda")
    h0, dh = normal(gen, b, h, dk, dv), normal(gen, b, h, dk, dv)

    def both(q, k, v, do):
        o, last = ss.lattn_fwd(q, k, v, decay, h0=h0, return_last_state=True)
        return {"o": o, "h_last": last, **ss.lattn_bwd(q, k, v, decay, do, h0=h0, dh_last=dh, want_dh0=True)}

    assert row.stride(0) > 1 << 20
    got, want = both(*views), both(*(t.contiguous() for t in views))
    # the same numbers, however the rows are read
    for n in want:
        assert torch.isfinite(want[n]).all() and torch.equal(got[n], want[n]), n
