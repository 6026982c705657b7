"""The gradients of the norms' weights on the GPU: sums over all tokens and heads, joined without losing bits."""
import pytest
import torch

from gpu_util import host64, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,heads,width,roundings", [
    (1000, 1, 512, 1),      # a workgroup has one head of one token: its sum is the term itself
    (1024, 1, 90, 1),
    (1024, 16, 96, 2),      # and 16 groups of lanes one head each: their sum is rounded, and the sum of those
    (517, 11, 57, 2),
    (3, 4, 256, 2),
])
def test_joined_sums(dtype, tokens, heads, width, roundings):
    """With x of ones, weights of ones and no rotation each term is dy itself, and with dy in [0.5, 1) every
    rounding counts, none cancelling: what is left is that of the workgroups' sums to fp32 and of the result."""
    import selective_state_space_85_amd as ss

    say("qknorm_bwd sums", dtype, tokens, heads, width)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(tokens)
    one = torch.ones((tokens, heads, width), dtype=dtype, device="cuda")
    w = torch.ones((width,), device="cuda")
    pos = torch.zeros((tokens,), dtype=torch.int64, device="cuda")
    inv = torch.empty((0,), device="cuda")
    dy = [(0.5 + 0.499 * torch.rand(one.shape, generator=gen, device="cuda")).to(dtype) for _ in range(2)]
    g = ss.qknorm_bwd(one, one, w, w, pos, inv, *dy, eps=0.0)
    torch.cuda.synchronize()
    for n, t in zip(("dw_q", "dw_k"), dy):
        want = host64(t).sum((0, 1))
        e = float((abs(host64(g[n]) - want) / want).max())
        say("   %s %.2e" % (n, e))
        assert e <= roundings * 2.0 ** -24 * (1 + 2.0 ** -20), (n, e)
