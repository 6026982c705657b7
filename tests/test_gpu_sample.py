"""Sampling on the GPU against its definition, row by row in 64 bits: tokens have to be equal."""
import numpy as np
import pytest
import torch

import attn_ref as ref
from gpu_util import host64, say

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ss():
    import selective_state_space_85_amd as ss

    assert torch.cuda.is_available()
    return ss


def f32(v):
    return float(np.float32(v))


def want(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    n = len(logits)
    rows = [host64(v) if isinstance(v, torch.Tensor) else np.full(n, f32(v)) for v in (u, temperature, top_k, top_p, min_p)]
    l = host64(logits)
    return [ref.sample_row(l[i], rows[0][i], rows[1][i], int(rows[2][i]), rows[3][i], rows[4][i]) for i in range(n)]


def logits(dtype, n, v, seed=0, std=2.5):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn((n, v), generator=gen, device="cuda") * std).to(dtype), torch.rand((n,), generator=gen, device="cuda")


SETTINGS = [
    dict(), dict(temperature=0.0), dict(temperature=0.7), dict(temperature=5.0), dict(temperature=0.01),
    dict(top_k=1), dict(top_k=50), dict(top_k=100000000), dict(top_p=0.9), dict(top_p=0.0), dict(top_p=1e-6),
    dict(top_p=0.999), dict(min_p=0.1), dict(min_p=1.0), dict(min_p=2.0), dict(temperature=0.8, top_k=40, top_p=0.95),
    dict(temperature=1.5, top_k=500, top_p=0.7, min_p=0.02), dict(temperature=-1.0, top_k=3),
    dict(temperature=float("inf"), top_p=0.5), dict(top_p=float("nan"), min_p=float("nan"), top_k=-7)]


@pytest.mark.parametrize("v", [1, 2, 63, 64, 1000, 5003, 50257])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_settings(ss, dtype, v):
    l, u = logits(dtype, 6, v, v)
    for kw in SETTINGS:
        say("sample", dtype, v, kw)
        got = ss.sample(l, u, **kw)
        assert got.dtype is torch.int64 and got.tolist() == want(l, u, **kw), kw


def test_settings_by_row(ss):
    say("sample by row")
    n = 300
    l, u = logits(F32, n, 3001, 1)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    r = lambda: torch.rand((n,), generator=gen, device="cuda")  # noqa: E731
    kw = dict(temperature=torch.where(r() < 0.2, 0.0, 0.3 + r()), top_k=(r() * 100).int(),
              top_p=torch.where(r() < 0.5, r(), 1.0), min_p=torch.where(r() < 0.5, 0.2 * r(), 0.0))
    assert ss.sample(l, u, **kw).tolist() == want(l, u, **kw)


@pytest.mark.parametrize("v", [7, 300, 4096, 6001, 131072])
def test_ties(ss, v):
    """Equal logits: the lowest index first, however many there are."""
    say("sample ties", v)
    u = torch.tensor([0.0, 0.25, 0.5, 0.75, 0.999999], device="cuda")
    flat = torch.full((5, v), -3.0, device="cuda")
    two = flat.clone()
    two[:, v // 2:] = -1.5
    zeros = torch.where(torch.arange(v, device="cuda") % 2 == 0, 0.0, -0.0).expand(5, v).contiguous()  # equal too
    steps = (torch.arange(v, device="cuda") % 5).float().flip(0).expand(5, v).contiguous()
    for l in (flat, two, zeros, steps, flat.bfloat16()):
        for kw in (dict(), dict(top_k=v // 2 + 1), dict(top_p=0.3), dict(temperature=0.0), dict(min_p=0.5),
                   dict(top_k=5, top_p=0.5, temperature=0.1)):
            assert ss.sample(l, u, **kw).tolist() == want(l, u, **kw), kw


def test_numbers_at_the_ends(ss):
    say("sample ends")
    u = torch.tensor([0.0, 0.5, 1.0, 2.0, -1.0, float("nan"), 1 - 2.0 ** -24, 2.0 ** -149], device="cuda")
    l, _ = logits(F32, 8, 777, 3)
    for kw in (dict(), dict(top_p=0.5), dict(top_k=3), dict(temperature=0.05)):
        assert ss.sample(l, u, **kw).tolist() == want(l, u, **kw), kw
    # logits near the type's ends, and temperatures that take their differences beyond it
    big = torch.tensor([[3.4e38, -3.4e38, 0.0, 3.4e38, 1e38]] * 8, device="cuda")
    for t in (1e-38, 1.0, 1e38, 3e38, 1e-45):
        assert ss.sample(big, u, temperature=t).tolist() == want(big, u, temperature=t), t
    tiny = torch.tensor([[1e-45, 0.0, -1e-45, 2e-45, 1e-38]] * 8, device="cuda")
    for t in (1e-45, 1e-44, 1.0):
        assert ss.sample(tiny, u, temperature=t).tolist() == want(tiny, u, temperature=t), t


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_where_the_largest_lie(ss, dtype):
    """The largest logits in a few threads' share of the row, in order, all equal, few that can be taken at all."""
    say("sample places", dtype)
    v = 20011
    l, u = logits(dtype, 8, v, 6)
    at = torch.arange(v, device="cuda")
    l[0, at % 8192 < 8] += 30.0
    l[1] = l[1].sort(descending=True).values
    l[2] = l[2].sort().values
    l[3, 900:] = -float("inf")
    l[4, 40:] = float("nan")
    l[5] = 1.25
    l[6, 100:] = 1.25
    l[7, :5000] = 9.0
    for k in (1, 2, 39, 41, 300, 895, 896, 897, 2000, 5000, 20010):
        for kw in (dict(), dict(temperature=0.2, top_p=0.9), dict(temperature=3.0, min_p=0.3)):
            assert ss.sample(l, u, top_k=k, **kw).tolist() == want(l, u, top_k=k, **kw), (k, kw)


def test_temperatures_beside_the_logits_steps(ss):
    """Temperatures from far below a step of the largest logit's to far above the logits' span."""
    say("sample steps")
    l, u = logits(F32, 6, 3000, 7)
    for scale in (1.0, 1e6, 1e12, 1e30):
        for t in (1e-30, 1e-3, 0.0625, 1.0, 1e6, 1e30, 3e38):
            for kw in (dict(), dict(top_k=20), dict(top_p=0.6)):
                x = l * scale + scale
                assert ss.sample(x, u, temperature=t, **kw).tolist() == want(x, u, temperature=t, **kw), (scale, t, kw)


def test_masked_logits(ss):
    """-infinity, the type's lowest value, +infinity and NaN; rows of which nothing is left."""
    say("sample masks")
    inf, nan = float("inf"), float("nan")
    for dtype in (F32, BF16):
        l, u = logits(dtype, 9, 500, 4)
        l[0] = -inf
        l[1] = nan
        l[2, 3:] = -inf
        l[3, ::2] = nan
        l[4, 7] = inf
        l[5, 100:103] = inf
        l[6] = -inf
        l[6, 499] = torch.finfo(dtype).min
        l[7, 1:] = torch.finfo(dtype).min
        l[8, 0:400] = torch.finfo(dtype).min
        l[8, 400:] = nan
        for kw in (dict(), dict(top_k=2), dict(top_p=0.6), dict(min_p=0.3), dict(temperature=0.0),
                   dict(temperature=0.3, top_k=4, top_p=0.8)):
            got = ss.sample(l, u, **kw).tolist()
            assert got == want(l, u, **kw), kw
            assert got[0] == got[1] == -1 and got[4] == 7 and got[6] == 499


def test_every_token_by_its_share(ss):
    """u over an even grid takes each token as often as its weight says, to one place."""
    say("sample shares")
    n = 4096
    l = torch.log(torch.tensor([0.5, 0.25, 0.125, 0.125], device="cuda")).expand(n, 4).contiguous()
    u = torch.arange(n, device="cuda").float() / n
    count = torch.bincount(ss.sample(l, u), minlength=4).tolist()
    assert all(abs(c - w * n) <= 1 for c, w in zip(count, (0.5, 0.25, 0.125, 0.125)))


def test_strided_rows_and_output(ss):
    say("sample strides")
    wide, u = logits(BF16, 5, 1100, 5)
    l = wide[:, 13:1000]
    out = torch.full((7,), 5, device="cuda")
    got = ss.sample(l, u, out=out[1:6])
    assert out.tolist() == [5] + want(l, u) + [5] and got.data_ptr() == out[1:6].data_ptr()
    assert ss.sample(l[:1], u[:1]).tolist() == want(l[:1], u[:1])


def test_refusals(ss):
    l, u = logits(F32, 4, 100, 6)
    with pytest.raises(TypeError):
        ss.sample(l.half(), u)
    with pytest.raises((TypeError, ValueError)):
        ss.sample(l, u.double())
    with pytest.raises((TypeError, ValueError)):
        ss.sample(l, u, top_k=torch.zeros((4,), dtype=torch.int64, device="cuda"))
    for bad in (dict(u=u[:3]), dict(temperature=torch.ones((3,), device="cuda")), dict(out=torch.empty((3,), dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError):
            ss.sample(l, **{"u": u, **bad})
    for bad in (l[0], l.t()[:, :4], l.cpu(), l[:0], l[:, :0]):
        with pytest.raises((ss.SSError, ValueError)):
            ss.sample(bad, u[:bad.shape[0]] if bad.dim() == 2 and bad.is_cuda else u)
