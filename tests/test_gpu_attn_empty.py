"""Tensors without elements are refused by linear attention, its norms and sampling, each as the other
operators refuse them; nothing runs on the GPU."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b,l,hk,h,dk,dv", [(0, 4, 1, 2, 8, 8), (2, 0, 1, 2, 8, 8), (2, 4, 0, 2, 8, 8), (2, 4, 1, 0, 8, 8),
                                            (2, 4, 1, 2, 0, 8), (2, 4, 1, 2, 8, 0)])
def test_attention(b, l, hk, h, dk, dv):
    import selective_state_space_85_amd as ss

    q, v = torch.zeros((b, l, hk, dk), device="cuda"), torch.zeros((b, l, h, dv), device="cuda")
    decay = torch.zeros((h,), device="cuda")
    for scale in (None, 0.5):
        with pytest.raises((ss.SSError, ValueError)):
            ss.lattn_fwd(q, q, v, decay, scale=scale)
        with pytest.raises((ss.SSError, ValueError)):
            ss.lattn_bwd(q, q, v, decay, v, scale=scale)
        if l:
            with pytest.raises((ss.SSError, ValueError)):
                ss.lattn_step(torch.zeros((b, h, dk, dv), device="cuda"), q[:, 0], q[:, 0], v[:, 0], decay, scale=scale)


@pytest.mark.parametrize("n,hq,hk,w", [(0, 1, 1, 8), (3, 0, 1, 8), (3, 1, 0, 8), (3, 1, 1, 0)])
def test_norms(n, hq, hk, w):
    import selective_state_space_85_amd as ss

    q, k, weight = torch.zeros((n, hq, w), device="cuda"), torch.zeros((n, hk, w), device="cuda"), torch.ones((w,), device="cuda")
    args = (q, k, weight, weight, torch.zeros((n,), dtype=torch.int64, device="cuda"), torch.zeros((0,), device="cuda"))
    with pytest.raises((ss.SSError, ValueError)):
        ss.qknorm_fwd(*args)
    with pytest.raises((ss.SSError, ValueError)):
        ss.qknorm_bwd(*args, q, k)


@pytest.mark.parametrize("n,v", [(0, 5), (5, 0)])
def test_sampling(n, v):
    import selective_state_space_85_amd as ss

    with pytest.raises((ss.SSError, ValueError)):
        ss.sample(torch.zeros((n, v), device="cuda"), torch.zeros((n,), device="cuda"))
