"""GPU: the gated linear recurrence at the lengths where its tiles, kept states and chunks begin and
end, and what it leaves of the memory behind its outputs."""
import numpy as np
import pytest
import torch

import lm_ref
import workloads as wl
from gpu_util import TOL, dev, host64, say
from test_gpu_glr import decays, make, rand, ss, tdev, wide, check

pytestmark = pytest.mark.gpu

ROWS = 320  # behind the last row: more than any tile has


def front(shape, dt, fill):
    """A tensor of `shape` at the front of a larger one full of `fill`, and what lies behind it."""
    n = int(np.prod(shape))
    whole = torch.full((n + ROWS * shape[-1],), fill, dtype=dt, device="cuda")
    return whole[:n].view(shape), whole[n:]


@pytest.mark.parametrize("dt", [wl.F32, wl.BF16])
@pytest.mark.parametrize("d", [64, 33, 70])
@pytest.mark.parametrize("l", [1, 3, 17, 33, 257])
def test_nothing_behind_the_last_row(l, d, dt):
    """Rows past the end are neither read (they hold NaN) nor written, of the last batch row either."""
    b = 2
    rng = np.random.default_rng(l + d)
    to = torch.bfloat16 if dt == wl.BF16 else torch.float32
    say("glr behind", l, d, dt)
    src = [dev(rand(rng, (b, l, d), dt)) for _ in range(4)]  # x, r, i, dy
    inp = []
    for s in src:
        t, _ = front((b, l, d), to, float("nan"))
        t.copy_(s)
        inp.append(t)
    decay = dev(decays(rng, d))
    reset = np.zeros((b, l), np.uint8)
    reset[:, l // 2] = 1
    for r in (None, tdev(reset)):
        y, y_rest = front((b, l, d), to, 7.0)
        ck, ck_rest = front(ss().glr_ckpt_shape(b, l, d), torch.float32, 7.0)
        hl, hl_rest = front((b, d), torch.float32, 7.0)
        g_out, g_rest = front((b, l, 3 * d), to, 7.0)
        ss().glr_fwd(*inp[:3], decay, reset=r, out=y, ckpt=ck, h_last=hl)
        g = ss().glr_bwd(*inp[:3], decay, inp[3], reset=r, ckpt=ck, out=g_out)
        ck2 = torch.empty_like(ck)
        y2, hl2 = ss().glr_fwd(*src[:3], decay, reset=r, ckpt=ck2, return_last_state=True)
        g2 = ss().glr_bwd(*src[:3], decay, src[3], reset=r, ckpt=ck2)
        torch.cuda.synchronize()
        for rest in (y_rest, ck_rest, hl_rest, g_rest):
            assert bool((rest == 7.0).all())
        assert torch.equal(y, y2) and torch.equal(ck, ck2) and torch.equal(hl, hl2)
        for n in g2:
            assert torch.equal(g[n], g2[n]) and bool(torch.isfinite(g[n]).all()), n


# batch, seqlen, dim, dtype, strided, h0, reset.  A forward tile has 256 rows, a backward tile and the
# rows between two kept states 32; the backward cuts the rows of fewer than 256 workgroups (batch times
# blocks of 64 channels) in chunks of at least 128 rows, at most 64 of them.
CASES = [
    (2, 32, 64, wl.F32, False, True, False),        # one backward tile exactly
    (1, 33, 66, wl.BF16, True, False, True),        # and one row more
    (1, 255, 64, wl.F32, False, True, True),        # one forward tile, one row short
    (2, 256, 70, wl.BF16, False, True, False),      # exactly; the first length of two chunks
    (1, 257, 33, wl.F32, True, False, True),        # two, the second of one row
    (1, 8192, 64, wl.F32, False, True, True),       # 64 chunks of 128 rows
    (1, 8193, 64, wl.BF16, True, False, False),     # the chunks' number bounded: 160 rows each
    (8, 300, 2050, wl.F32, False, True, False),     # 264 workgroups: rows uncut, ten backward tiles
    (8, 300, 2050, wl.BF16, True, True, True),
    (32, 520, 512, wl.BF16, False, False, True),    # 256 workgroups, even channels
]
IDS = ["B%dL%dD%d-%s%s%s%s" % (c[0], c[1], c[2], c[3], "-str" * c[4], "-h0" * c[5], "-reset" * c[6]) for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_lengths(case):
    b, l, d, dt = case[:4]
    p = make(case, 300)
    say("glr lengths", case)
    x, r, i = p["t"]
    kw = dict(h0=tdev(p["h0"]), reset=tdev(p["reset"]))
    ck = torch.full(ss().glr_ckpt_shape(b, l, d), float("nan"), device="cuda")
    y, hl = ss().glr_fwd(x, r, i, dev(p["decay"]), return_last_state=True, ckpt=ck, **kw)
    g = ss().glr_bwd(x, r, i, dev(p["decay"]), dev(p["dy"]), ckpt=ck, dh_last=tdev(p["dh_last"]), **kw)
    g2 = ss().glr_bwd(x, r, i, dev(p["decay"]), dev(p["dy"]), dh_last=tdev(p["dh_last"]), **kw)
    torch.cuda.synchronize()
    decay = p["decay"].astype(np.float64)
    yr, hr = lm_ref.glr(*p["ref"], decay, 8.0, p["h0"], p["reset"])
    check("y", host64(y), yr, TOL[dt])
    check("h_last", host64(hl), hr, TOL["f32"])
    ref = lm_ref.glr_bwd(*p["ref"], decay, 8.0, wide(p["dy"]), p["h0"], p["reset"], p["dh_last"])
    for n in ref:
        check(n, host64(g[n]), ref[n], TOL["f32"] if n in ("ddecay", "dh0") else TOL[dt])
        assert torch.equal(g2[n], g[n]), n


def test_the_largest_launch():
    """As many sequences as one launch takes (2^32 threads less one workgroup's), and one more refused."""
    b, d = (1 << 23) - 1, 2
    gen = torch.Generator(device="cuda").manual_seed(3)
    say("glr largest launch")
    x, r, i = ((torch.randn((b + 1, 1, d), generator=gen, device="cuda")).bfloat16() for _ in range(3))
    decay = torch.tensor([-2.0, 0.5], device="cuda")
    y = ss().glr_fwd(x[:b], r[:b], i[:b], decay)
    h = torch.zeros((b, d), device="cuda")
    ys = ss().glr_step(h, x[:b, 0], r[:b, 0], i[:b, 0], decay)
    torch.cuda.synchronize()
    assert torch.equal(y[:, 0], ys)
    with pytest.raises(ss().SSError, match="UNSUPPORTED"):
        ss().glr_fwd(x, r, i, decay)
