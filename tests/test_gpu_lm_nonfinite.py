"""GPU: operands of the largest and smallest magnitudes, infinities and NaN in the language-model
operators, in every way that a product or a recurrence is formed."""
import numpy as np
import pytest
import torch

import lm_ref
import workloads as wl
from gpu_util import TOL, dev, host64, say
from test_gpu_glr import check, rand, wide

pytestmark = pytest.mark.gpu

TOP = np.finfo(np.float32).max


def ss():
    import selective_state_space_85_amd as m

    return m


def same(name, got, ref, bar):
    """NaN and infinities where the definition has them, and the rest within the bar."""
    assert np.array_equal(np.isnan(got), np.isnan(ref)), name
    inf = np.isinf(ref)
    assert np.array_equal(np.isinf(got), inf) and np.array_equal(got[inf], ref[inf]), name
    ok = np.isfinite(ref)
    check(name, np.where(ok, got, 0.0), np.where(ok, ref, 0.0), bar)


# rows: gradients in one pass over the weights; streamed past them; 64 x 128 tiles; 128 x 128 tiles
XENT = [(3, 40, 700), (12, 40, 700), (200, 40, 700), (1024, 33, 4096)]


def xent_case(n, d, v, seed=0):
    rng = np.random.default_rng(seed + n)
    x = rng.standard_normal((n, d)).astype(np.float32)
    w = (rng.standard_normal((v, d)) * 2 / np.sqrt(d)).astype(np.float32)
    t = rng.integers(0, v, n)
    dloss = rng.uniform(0.1, 1.0, n).astype(np.float32)
    return x, w, t, dloss


def xent(x, w, t, dloss):
    tt = torch.from_numpy(t).cuda()
    loss, lse = ss().xent_fwd(dev(x), dev(w), tt)
    g = ss().xent_bwd(dev(x), dev(w), tt, lse, dev(dloss))
    torch.cuda.synchronize()
    return host64(loss), host64(lse), {k: host64(q) for k, q in g.items()}


@pytest.mark.parametrize("n,d,v", XENT)
@pytest.mark.parametrize("mask", [-TOP, -np.inf], ids=["lowest", "-inf"])
def test_masked_entries(n, d, v, mask):
    """A bias folded into w masks a part of the vocabulary, a whole group of 128 entries among it:
    those entries count as nothing."""
    x, w, t, dloss = xent_case(n, d, v)
    x[:, 3] = 1.0
    out = np.zeros(v, bool)
    out[5:v:7] = True
    out[128:256] = True
    w[:, 3] = np.where(out, mask, 0.0)
    t = np.flatnonzero(~out)[t % (~out).sum()]
    say("xent mask", n, d, v, mask)
    loss, lse, g = xent(x, w, t, dloss)
    x64, w64 = x.astype(np.float64), w.astype(np.float64)
    keep = x64 @ w64[~out].T
    top = keep.max(1)
    zr = top + np.log(np.exp(keep - top[:, None]).sum(1))
    check("lse", lse, zr, TOL["f32"])
    check("loss", loss, zr - (x64 * w64[t]).sum(1), TOL["f32"])
    p = np.zeros((n, v))
    p[:, ~out] = np.exp(keep - zr[:, None])
    p[np.arange(n), t] -= 1.0
    p *= dloss[:, None].astype(np.float64)
    check("dw", g["dw"], p.T @ x64, TOL["f32"])
    dx = p[:, ~out] @ w64[~out]
    cols = np.arange(d) != 3
    check("dx", g["dx"][:, cols], dx[:, cols], TOL["f32"])
    # 0 times the mask itself: 0, or NaN where that is infinite
    want = np.isinf(mask)
    assert np.all(np.isnan(g["dx"][:, 3]) == want) and (want or not g["dx"][:, 3].any())


@pytest.mark.parametrize("n,d,v", XENT)
def test_largest_finite_operands(n, d, v):
    """x of the largest magnitude beside weights of 0: nothing of it in the logits, and a finite dw."""
    x, w, t, dloss = xent_case(n, d, v, 1)
    w[:, 2] = 0.0
    x[1::3, 2], x[2::3, 2] = TOP, -TOP
    dloss *= np.float32(2.0 ** -100)
    say("xent largest", n, d, v)
    loss, lse, g = xent(x, w, t, dloss)
    x64, w64 = x.astype(np.float64), w.astype(np.float64)
    lr, zr, _, _ = lm_ref.xent(x64, w64, t)
    check("loss", loss, lr, TOL["f32"])
    check("lse", lse, zr, TOL["f32"])
    ref = lm_ref.xent_bwd(x64, w64, t, dloss.astype(np.float64))
    check("dx", g["dx"] * 2.0 ** 100, ref["dx"] * 2.0 ** 100, TOL["f32"])
    cols = np.arange(d) != 2
    check("dw", g["dw"][:, cols] * 2.0 ** 100, ref["dw"][:, cols] * 2.0 ** 100, TOL["f32"])
    # the products of dl with x's largest values
    check("dw", g["dw"][:, 2] * 2.0 ** -28, ref["dw"][:, 2] * 2.0 ** -28, TOL["f32"])


@pytest.mark.parametrize("m", [12, 40, 200, 1100])
def test_projection_of_large_and_tiny(m):
    """Pre-activations from x at the largest magnitude, and from x of 1e-36.  In tiles an operand's
    parts end at 2^-134, which is 4.6e-5 of 1e-36: at most twice that in a product of two such sums."""
    k, f = 48, 1000
    rng = np.random.default_rng(m)
    x = rng.standard_normal((m, k)).astype(np.float32)
    wg, wu = ((rng.standard_normal((f, k)) / np.sqrt(k)).astype(np.float32) for _ in range(2))
    x[:, 0] = np.where(np.arange(m) % 2, TOP, -TOP)
    wg[:, 0] = rng.uniform(1.0, 2.0, f) * 2.0 ** -122
    wu[:, 0] = 0.0
    say("glu large", m)
    h = host64(ss().glu_fwd(dev(x), dev(wg), dev(wu)))
    p = [v.astype(np.float64) for v in (x, wg, wu)]
    # 2^-134 of wg's first column times 2^128: 2^-6 of 64 and more, 2.5e-4
    check("h", h, lm_ref.glu(*p, "silu"), 5e-4)
    x = (rng.uniform(1.0, 1.9, (m, k)) * 1e-36).astype(np.float32)
    wg, wu = ((rng.uniform(0.5, 1.0, (f, k)) * s).astype(np.float32) for s in (1e36, 2e35))
    say("glu tiny", m)
    h = host64(ss().glu_fwd(dev(x), dev(wg), dev(wu)))
    check("h", h, lm_ref.glu(*[v.astype(np.float64) for v in (x, wg, wu)], "silu"), TOL["f32"])


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("m", [12, 40, 200, 1100])
def test_projection_of_infinities(m, act):
    """An infinite token and an infinite weight give what IEEE products and sums of them are,
    however many tokens share the call; gradients too."""
    k, f = 48, 1000
    rng = np.random.default_rng(m + 1)
    x = rng.standard_normal((m, k)).astype(np.float32)
    wg, wu = ((rng.standard_normal((f, k)) / np.sqrt(k)).astype(np.float32) for _ in range(2))
    dh = rng.standard_normal((m, f)).astype(np.float32)
    x[7, 5], x[9, 40], x[11, 2] = np.inf, -np.inf, np.nan
    wu[21, 8] = np.inf
    say("glu inf", m, act)
    t = [dev(v) for v in (x, wg, wu)]
    h = ss().glu_fwd(*t, act=act)
    torch.cuda.synchronize()
    p = [v.astype(np.float64) for v in (x, wg, wu)]
    with np.errstate(all="ignore"):
        same("h", host64(h), lm_ref.glu(*p, act), TOL["f32"])
        # gradients: of finite tokens, the weight alone infinite (in the product's transposed operand)
        x[7, 5] = x[9, 40] = x[11, 2] = 0.25
        p[0] = x.astype(np.float64)
        g = ss().glu_bwd(dev(x), *t[1:], dev(dh), act=act)
        torch.cuda.synchronize()
        ref = lm_ref.glu_bwd(*p, dh.astype(np.float64), act)
        for n in ref:
            same(n, host64(g[n]), ref[n], TOL["f32"])


@pytest.mark.parametrize("m,k,f", [(200, 40, 700), (1100, 48, 1000)])
def test_neighbours_keep_their_bits(m, k, f):
    """fp32 in tiles: a NaN and an infinite token change nothing of the others, to the bit."""
    rng = np.random.default_rng(m)
    x = rng.standard_normal((m, k)).astype(np.float32)
    w, w2 = ((rng.standard_normal((f, k)) / np.sqrt(k)).astype(np.float32) for _ in range(2))
    bad = x.copy()
    bad[17, 3], bad[131, 5] = np.nan, np.inf
    rows = np.ones(m, bool)
    rows[[17, 131]] = False
    at = torch.from_numpy(np.flatnonzero(rows)).cuda()
    t = torch.from_numpy(rng.integers(0, f, m)).cuda()
    dh, dloss = dev(rng.standard_normal((m, f)).astype(np.float32)), torch.ones(m, device="cuda")
    say("neighbours", m, k, f)

    def both(xs):
        xt = dev(xs)
        loss, lse = ss().xent_fwd(xt, dev(w), t)
        return (ss().glu_fwd(xt, dev(w), dev(w2)), ss().glu_bwd(xt, dev(w), dev(w2), dh)["dx"], loss, lse,
                ss().xent_bwd(xt, dev(w), t, lse, dloss)["dx"])

    for got, want in zip(both(bad), both(x)):
        assert torch.equal(got[at], want[at])
        assert not bool(torch.isfinite(got[17]).any())


# decays so fast that the product of a over a few rows lies below float32's range: nothing of a
# NaN or an infinity is lost with it
@pytest.mark.parametrize("dt", [wl.F32, wl.BF16])
@pytest.mark.parametrize("l,d", [(40, 33), (700, 64)])
@pytest.mark.parametrize("with_reset", [False, True], ids=["no-resets", "resets-elsewhere"])
@pytest.mark.parametrize("what", [np.nan, np.inf], ids=["nan", "inf"])
def test_fast_decays_keep_nonfinite_states(what, with_reset, l, d, dt):
    rng = np.random.default_rng(l)
    b = 2
    v = [rand(rng, (b, l, d), dt) for _ in range(3)]
    w = [wide(a).astype(np.float32) for a in v]
    w[0][0, 5, 7] = what
    t = [torch.from_numpy(a).cuda().to(torch.bfloat16 if dt == wl.BF16 else torch.float32) for a in w]
    decay = np.full(d, 2.0, np.float32)  # k = 17, a about e^-8.5
    reset = None
    if with_reset:
        reset = np.zeros((b, l), np.uint8)
        reset[1, 17] = 1  # the other batch row's
    say("glr fast", what, with_reset, l, d, dt)
    y, hl = ss().glr_fwd(*t, dev(decay), reset=None if reset is None else torch.from_numpy(reset).cuda(),
                         return_last_state=True)
    torch.cuda.synchronize()
    y, hl = host64(y), host64(hl)
    bad = np.zeros((b, l, d), bool)
    bad[0, 5:, 7] = True
    assert np.array_equal(~np.isfinite(y), bad)
    assert np.all(np.isnan(y[bad])) if np.isnan(what) else np.all(y[bad] == what)
    assert np.array_equal(~np.isfinite(hl), bad[:, -1])
    # backward: a NaN among dy reaches every row before it
    dy = np.zeros((b, l, d), np.float32)
    dy[0, l - 2, 9] = np.nan
    w[0][0, 5, 7] = 0.0
    t[0] = torch.from_numpy(w[0]).cuda().to(t[0].dtype)
    g = ss().glr_bwd(*t, dev(decay), torch.from_numpy(dy).cuda().to(t[0].dtype),
                     reset=None if reset is None else torch.from_numpy(reset).cuda())
    torch.cuda.synchronize()
    bad[:] = False
    bad[0, :l - 1, 9] = True
    for n in ("dx", "dr", "di"):
        assert np.array_equal(np.isnan(host64(g[n])), bad), n
    assert np.array_equal(np.isnan(host64(g["dh0"])), bad[:, 0])
    assert np.array_equal(np.isnan(host64(g["ddecay"])), bad[0, 0])


@pytest.mark.parametrize("dt", [wl.F32, wl.BF16])
@pytest.mark.parametrize("l,d", [(40, 33), (700, 64)])
def test_a_reset_ends_nonfinite_states_of_fast_decays(l, d, dt):
    """A reset cuts a NaN off on both sides: from the states after it, and from the gradients of
    the rows before it."""
    rng = np.random.default_rng(l + 1)
    b, at = 2, l // 2
    w = [wide(rand(rng, (b, l, d), dt)).astype(np.float32) for _ in range(3)]
    w[0][0, 5, 7] = np.nan
    to = torch.bfloat16 if dt == wl.BF16 else torch.float32
    t = [torch.from_numpy(a).cuda().to(to) for a in w]
    decay = dev(np.full(d, 2.0, np.float32))
    reset = np.zeros((b, l), np.uint8)
    reset[0, at] = 1
    r = torch.from_numpy(reset).cuda()
    say("glr fast reset", l, d, dt)
    y = host64(ss().glr_fwd(*t, decay, reset=r))
    bad = np.zeros((b, l, d), bool)
    bad[0, 5:at, 7] = True
    assert np.array_equal(np.isnan(y), bad)
    w[0][0, 5, 7] = 0.0
    t[0] = torch.from_numpy(w[0]).cuda().to(to)
    dy = np.zeros((b, l, d), np.float32)
    dy[0, l - 2, 9] = np.nan
    g = ss().glr_bwd(*t, decay, torch.from_numpy(dy).cuda().to(to), reset=r)
    torch.cuda.synchronize()
    bad[:] = False
    bad[0, at:l - 1, 9] = True
    for n in ("dx", "di"):
        assert np.array_equal(np.isnan(host64(g[n])), bad), n
    bad[0, at] = False  # the reset row's a is 0 whatever its gate
    assert np.array_equal(np.isnan(host64(g["dr"])), bad)
    assert not np.isnan(host64(g["dh0"])).any()
