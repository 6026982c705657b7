"""GPU parity of the gated feed-forward projection (ss_glu_fwd, ss_glu_bwd) with its float64
definition.  fp32: <= 1e-4 max relative error.  bf16: <= 2e-2: outputs are rounded once, the
gradients of the two products once more between the products (2^-9 relative each)."""
import numpy as np
import pytest
import torch

import lm_ref
import workloads as wl
from gpu_util import TOL, dev, host64, rel_err, say
from test_gpu_glr import check, rand, wide

pytestmark = pytest.mark.gpu


def ss():
    import selective_state_space_85_amd as m

    return m


def make(m, k, f, dt, seed, extra=0):
    rng = np.random.default_rng(seed + 31 * m + 7 * k + f)
    x = rand(rng, (m, k + extra), dt)
    wg, wu = (rand(rng, (f, k), dt, 1.0 / np.sqrt(k)) for _ in range(2))
    dh = rand(rng, (m, f), dt)
    return x, wg, wu, dh


# tokens, dim, features, dtype, act, extra columns of x's rows
CASES = [
    (1, 1, 1, wl.F32, "silu", 0),
    (1, 8, 8, wl.BF16, "silu", 0),
    (1, 640, 200, wl.BF16, "gelu", 0),
    (1, 100, 33, wl.F32, "silu", 0),
    (5, 96, 130, wl.BF16, "silu", 8),
    (16, 257, 64, wl.BF16, "gelu", 0),        # dim in no whole 16 bytes: padded copies
    (17, 264, 40, wl.BF16, "silu", 0),
    (33, 512, 96, wl.F32, "gelu", 4),
    (64, 1032, 70, wl.BF16, "silu", 0),       # the last streamed row count
    (65, 200, 129, wl.BF16, "silu", 0),       # the first tiled one
    (130, 72, 257, wl.F32, "gelu", 0),
    (200, 333, 65, wl.F32, "silu", 3),
    (300, 136, 515, wl.BF16, "gelu", 24),
    (257, 320, 1000, wl.BF16, "silu", 0),
    # few tokens and many features: dx's sums are cut in parts (2, 62, and more than there are k tiles for)
    (40, 64, 1030, wl.BF16, "silu", 0),
    (3, 40, 16000, wl.F32, "silu", 0),
    (1, 16, 20510, wl.BF16, "gelu", 0),
    # many tokens and few features: the weights' sums are cut in parts
    (5000, 40, 33, wl.BF16, "silu", 0),
    (4100, 24, 20, wl.F32, "gelu", 0),
]
IDS = ["M%dK%dF%d-%s-%s%s" % (c[0], c[1], c[2], c[3], c[4], "-str" * (c[5] > 0)) for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward_and_gradients(case):
    m, k, f, dt, act, extra = case
    x, wg, wu, dh = make(m, k, f, dt, 1, extra)
    say("glu", case)
    xt, g_, u_ = dev(x)[:, :k], dev(wg), dev(wu)
    h = ss().glu_fwd(xt, g_, u_, act=act)
    g = ss().glu_bwd(xt, g_, u_, dev(dh), act=act)
    torch.cuda.synchronize()
    x64, wg64, wu64, dh64 = wide(x)[:, :k], wide(wg), wide(wu), wide(dh)
    check("h", host64(h), lm_ref.glu(x64, wg64, wu64, act), TOL[dt])
    ref = lm_ref.glu_bwd(x64, wg64, wu64, dh64, act)
    for n in ref:
        check(n, host64(g[n]), ref[n], TOL[dt])
    # each set of gradients alone
    only = ss().glu_bwd(xt, g_, u_, dev(dh), act=act, want_dw=False)
    assert set(only) == {"dx"} and torch.equal(only["dx"], g["dx"])
    only = ss().glu_bwd(xt, g_, u_, dev(dh), act=act, want_dx=False)
    assert set(only) == {"dw_gate", "dw_up"} and torch.equal(only["dw_up"], g["dw_up"])


@pytest.mark.parametrize("m,k,f", [(2200, 512, 1152), (4096, 264, 520)])
def test_large_tiles(m, k, f):
    """Enough tiles for the 256 x 256 ones, ragged in every direction."""
    x, wg, wu, dh = make(m, k, f, wl.BF16, 2)
    say("glu large", m, k, f)
    t = [dev(v) for v in (x, wg, wu)]
    h = ss().glu_fwd(*t)
    g = ss().glu_bwd(*t, dev(dh))
    torch.cuda.synchronize()
    p = [wide(v) for v in (x, wg, wu)]
    check("h", host64(h), lm_ref.glu(*p, "silu"), TOL["bf16"])
    ref = lm_ref.glu_bwd(*p, wide(dh), "silu")
    for n in ref:
        check(n, host64(g[n]), ref[n], TOL["bf16"])


@pytest.mark.parametrize("m", [3, 40, 150])
def test_fp32_rows_off_any_boundary(m):
    """fp32 takes operands that start off a 16-byte boundary with an odd row stride."""
    k, f = 64, 70
    x, wg, wu, dh = make(m, k, f, wl.F32, 9, 5)
    xt = dev(np.concatenate([np.zeros((m, 2), np.float32), x[:, :k + 1]], 1))[:, 3:3 + k]
    flat = dev(np.concatenate([[0.0], wg.reshape(-1)]).astype(np.float32))
    g_ = flat[1:].view(f, k)
    say("glu fp32 unaligned", m)
    h = ss().glu_fwd(xt, g_, dev(wu))
    g = ss().glu_bwd(xt, g_, dev(wu), dev(dh))
    torch.cuda.synchronize()
    x64 = wide(x)[:, 1:1 + k]
    check("h", host64(h), lm_ref.glu(x64, wide(wg), wide(wu), "silu"), TOL["f32"])
    ref = lm_ref.glu_bwd(x64, wide(wg), wide(wu), wide(dh), "silu")
    for n in ref:
        check(n, host64(g[n]), ref[n], TOL["f32"])


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activation_extremes(act):
    """Pre-activations from -1e4 to 1e4: the activation and its slope neither overflow nor
    lose their limits."""
    k = 8
    x = np.zeros((9, k), np.float32)
    x[:, 0] = [-1e4, -200.0, -90.0, -20.0, 0.0, 20.0, 90.0, 200.0, 1e4]
    x[:, 1] = 1.0
    wg, wu = np.zeros((4, k), np.float32), np.zeros((4, k), np.float32)
    wg[:, 0] = [1.0, 0.5, 0.01, -1.0]
    wu[:, 1] = 1.0
    dh = np.ones((9, 4), np.float32)
    say("glu extremes", act)
    t = [dev(v) for v in (x, wg, wu)]
    h = ss().glu_fwd(*t, act=act)
    g = ss().glu_bwd(*t, dev(dh), act=act)
    torch.cuda.synchronize()
    p = [v.astype(np.float64) for v in (x, wg, wu)]
    check("h", host64(h), lm_ref.glu(*p, act), TOL["f32"])
    ref = lm_ref.glu_bwd(*p, dh.astype(np.float64), act)
    for n in ref:
        check(n, host64(g[n]), ref[n], TOL["f32"])


def test_gradient_against_differences():
    m, k, f = 3, 4, 5
    x, wg, wu, dh = make(m, k, f, wl.F32, 3)
    say("glu differences")
    g = ss().glu_bwd(dev(x), dev(wg), dev(wu), dev(dh), act="gelu")
    torch.cuda.synchronize()
    inp = {"dx": x, "dw_gate": wg, "dw_up": wu}
    for name, arr in inp.items():
        num = np.zeros(arr.shape)
        for at in np.ndindex(arr.shape):
            v = []
            for s in (1e-5, -1e-5):
                q = {n: w.astype(np.float64) for n, w in inp.items()}
                q[name][at] += s
                v.append((lm_ref.glu(q["dx"], q["dw_gate"], q["dw_up"], "gelu") * dh).sum())
            num[at] = (v[0] - v[1]) / 2e-5
        check(name, host64(g[name]), num, TOL["f32"])


def test_a_tokens_result_does_not_depend_on_its_neighbours():
    """A NaN or infinite token stays in its own row."""
    x, wg, wu, _ = make(200, 64, 96, wl.BF16, 4)
    x32 = wl.bf16_bits_to_f32(x).copy()
    x32[17, 3], x32[131, 5] = np.nan, np.inf
    t = torch.from_numpy(x32).cuda().bfloat16()
    say("glu nan rows")
    h = host64(ss().glu_fwd(t, dev(wg), dev(wu)))
    clean = host64(ss().glu_fwd(dev(x), dev(wg), dev(wu)))
    rows = np.ones(200, bool)
    rows[[17, 131]] = False
    assert np.array_equal(h[rows], clean[rows]) and np.all(~np.isfinite(h[[17, 131]]).any(1))


def test_refusals():
    m = ss()
    x, w = torch.zeros((4, 64), device="cuda"), torch.zeros((32, 64), device="cuda")
    with pytest.raises(ValueError):
        m.glu_fwd(x, w, w[:16])
    with pytest.raises(ValueError):
        m.glu_fwd(x, w, w, act="relu")
    with pytest.raises(TypeError):
        m.glu_fwd(x.half(), w.half(), w.half())
    with pytest.raises(TypeError):
        m.glu_fwd(x, w.bfloat16(), w.bfloat16())
    with pytest.raises(ValueError):
        m.glu_fwd(x.t().contiguous().t(), w, w)
    with pytest.raises(m.SSError):  # bf16 rows that start off a 16-byte boundary
        m.glu_fwd(torch.zeros((4, 67), device="cuda").bfloat16()[:, 3:], w.bfloat16(), w.bfloat16())
    with pytest.raises(m.SSError):
        m.glu_bwd(x, w, w, torch.zeros((4, 32), device="cuda"), want_dx=False, want_dw=False)
    with pytest.raises(m.SSError):
        m.glu_bwd(x, w, w, torch.zeros((4, 32), device="cuda"),
                  workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("m,k,f", [(3, 2048, 4200), (4, 1032, 16450), (9, 256, 16500), (64, 136, 2600)],
                         ids=["one-pass", "one-pass-beside-tiles", "tiles", "streamed"])
def test_few_tokens_of_large_weights(m, k, f):
    """bf16, a few tokens: each way that the products and their gradients are formed."""
    x, wg, wu, dh = make(m, k, f, wl.BF16, 11)
    say("glu few", m, k, f)
    t = [dev(v) for v in (x, wg, wu)]
    h = ss().glu_fwd(*t)
    g = ss().glu_bwd(*t, dev(dh))
    torch.cuda.synchronize()
    p = [wide(v) for v in (x, wg, wu)]
    check("h", host64(h), lm_ref.glu(*p, "silu"), TOL["bf16"])
    ref = lm_ref.glu_bwd(*p, wide(dh), "silu")
    for n in ref:
        check(n, host64(g[n]), ref[n], TOL["bf16"])
