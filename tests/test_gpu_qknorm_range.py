"""Norms of queries and keys on the GPU where the squares leave fp32's range."""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("width", [64, 90, 7])
def test_squares_out_of_range(dtype, width):
    """Heads of 1e20 are normed to 0, of 1e-25 by eps alone, of zeros and those to what is not finite without
    an eps; ordinary heads beside them as ever."""
    import selective_state_space_85_amd as ss

    say("qknorm range", dtype, width)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(width)
    x = torch.randn((4, 1, width), generator=gen, device="cuda").to(dtype)
    dy = torch.randn((4, 1, width), generator=gen, device="cuda").to(dtype)
    sign = torch.where(torch.arange(width, device="cuda") % 2 == 0, 1.0, -1.0)
    x[1], x[2], x[3] = (1e20 * sign).to(dtype), (1e-25 * sign).to(dtype), 0.0
    w = torch.ones((width,), device="cuda")
    args = (w, w, torch.zeros((4,), dtype=torch.int64, device="cuda"), torch.empty((0,), device="cuda"))
    for eps in (0.0, 1e-4):
        y, _ = ss.qknorm_fwd(x, x, *args, eps=eps)
        g = ss.qknorm_bwd(x, x, *args, dy, dy, eps=eps)["dq"]
        first = ss.qknorm_fwd(x[:1], x[:1], *args[:2], args[2][:1], args[3], eps=eps)[0]
        assert torch.equal(y[:1], first) and torch.isfinite(first).all() and torch.isfinite(g[0]).all()
        assert (y[1] == 0).all() and (g[1] == 0).all()
        if eps:
            # by 1 / sqrt(eps): the root's and the product's roundings in fp32 and, in bf16, the output's
            want = x[2].double() * eps ** -0.5
            assert ((y[2].double() - want).abs() <= want.abs() * (4 * 2.0 ** -24 + (2.0 ** -8 if dtype is torch.bfloat16 else 0))).all()
            assert (y[3] == 0).all() and torch.isfinite(g[2:]).all()
        else:
            assert not torch.isfinite(y[2]).any() and torch.isnan(y[3]).all()
