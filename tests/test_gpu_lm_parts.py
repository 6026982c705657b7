"""GPU: sums of the matrix operators' gradients that are cut in parts, and the cross entropy's target
remainders where most targets are the same few."""
import numpy as np
import pytest
import torch

import lm_ref
import workloads as wl
from gpu_util import TOL, dev, host64, say
from test_gpu_glr import check, rand, wide

pytestmark = pytest.mark.gpu


def ss():
    import selective_state_space_85_amd as m

    return m


# tokens, dim, features.  fp32 beyond 8 tokens: dx's sums over 2 x features in tiles, cut into parts
# of at least 16 k tiles of 32 (62 and 6 of them, 11, 6); the last: the weights' sums over the tokens in 62
@pytest.mark.parametrize("m,k,f", [(12, 40, 16000), (777, 33, 2731), (40, 33, 3000), (64, 130, 1600), (32000, 36, 10)])
def test_fp32_projection_gradients_in_parts(m, k, f):
    rng = np.random.default_rng(m + k)
    x, dh = rand(rng, (m, k), wl.F32), rand(rng, (m, f), wl.F32)
    wg, wu = (rand(rng, (f, k), wl.F32, 1.0 / np.sqrt(k)) for _ in range(2))
    say("glu fp32 parts", m, k, f)
    t = [dev(v) for v in (x, wg, wu)]
    h = ss().glu_fwd(*t, act="gelu")
    g = ss().glu_bwd(*t, dev(dh), act="gelu")
    again = ss().glu_bwd(*t, dev(dh), act="gelu")
    torch.cuda.synchronize()
    p = [wide(v) for v in (x, wg, wu)]
    check("h", host64(h), lm_ref.glu(*p, "gelu"), TOL["f32"])
    ref = lm_ref.glu_bwd(*p, wide(dh), "gelu")
    for n in ref:
        check(n, host64(g[n]), ref[n], TOL["f32"])
        assert torch.equal(g[n], again[n]), n


# targets: all in one group of 128 entries (a mini tile is half of it), or on both sides of a bound
@pytest.mark.parametrize("n,d,v", [(300, 72, 500), (2304, 264, 8192), (4000, 40, 20001)])
@pytest.mark.parametrize("where", [(5, 9), (120, 136), (250, 262)])
def test_many_tokens_of_few_targets(n, d, v, where):
    rng = np.random.default_rng(n + where[0])
    x = dev(rand(rng, (n, d), wl.BF16))
    w = dev(rand(rng, (v, d), wl.BF16, 2.0 / np.sqrt(d)))
    t = torch.from_numpy(rng.integers(where[0], where[1], n)).cuda()
    t[::17] = v - 1
    dloss = torch.from_numpy(rng.uniform(0.1, 1.0, n)).cuda().float()
    say("xent few targets", n, d, v, where)
    loss, lse = ss().xent_fwd(x, w, t)
    g = ss().xent_bwd(x, w, t, lse, dloss)
    torch.cuda.synchronize()
    x64, w64, at = x.double(), w.double(), torch.arange(n, device="cuda")
    logits = torch.mm(x64, w64.t().contiguous())
    z = torch.logsumexp(logits, 1)
    check("loss", host64(loss), (z - logits[at, t]).cpu().numpy(), TOL["f32"])
    p = (logits - z[:, None]).exp()
    p[at, t] -= 1.0
    p *= dloss.double()[:, None]
    check("dx", host64(g["dx"]), torch.mm(p, w64).cpu().numpy(), TOL["bf16"])
    check("dw", host64(g["dw"]), torch.mm(p.t().contiguous(), x64).cpu().numpy(), TOL["bf16"])
