"""GPU: what the roundings of linear attention leave, in the root mean square, and rows read element by
element where a sequence is cut in segments.

bf16: rounding a number to 8 bits errs by 2^-7 / sqrt(12) of its binade, 0.00166 of the number in the mean
square over evenly spread mantissas.  Each of an output's terms has one factor that is rounded, the state or
a product of two rows, each by as much and independently, so that the sum errs by 0.00166 of its root mean
square too, and the output's own rounding makes it 0.00235.  A third rounding would make it 0.00287; the bar
is 8% above 0.00235.

fp32: a product's three parts leave out less than 2^-23 of it.  Every matrix instruction rounds the sum so far
by up to 2^-24 of it, six of them for each 16 terms; a sum of terms of mixed signs is sqrt(i) of them large
after i, so n roundings leave sqrt(n / 2) of one."""
import numpy as np
import pytest
import torch

import attn_ref as ref
from gpu_util import host64, say
from test_gpu_lattn import BF16, F32, check, make, numbers

pytestmark = pytest.mark.gpu

TWICE = 0.00254


def run(args, extra, do, dh, scale):
    import selective_state_space_85_amd as ss

    o, last = ss.lattn_fwd(**args, **extra, scale=scale, return_last_state=True)
    g = ss.lattn_bwd(**args, **extra, do=do, dh_last=dh, want_dh0=True, scale=scale)
    torch.cuda.synchronize()
    a, e = numbers(args, extra)
    want_o, want_last = ref.lattn(**a, scale=scale, **e)
    want = ref.lattn_bwd(**a, **e, scale=scale, do=host64(do), dh_last=None if dh is None else host64(dh))
    return {"o": o, "h_last": last, **g}, {"o": want_o, "h_last": want_last, **want}


#  type  b  l   hk h  dk   dv   reset  sliced
PRECISE = [
    (BF16, 2, 300, 2, 2, 128, 128, None, 0),
    (BF16, 2, 300, 1, 4, 64, 64, 0.01, 0),      # shared: sums of four heads' parts, in fp32
    (BF16, 1, 1500, 1, 2, 128, 64, None, 0),    # in segments; gradients in two launches
    (BF16, 1, 1500, 1, 2, 64, 128, 0.002, 0),
    (BF16, 1, 300, 1, 1, 256, 256, None, 0),
    (BF16, 2, 300, 1, 2, 125, 127, 0.01, 1),    # at any address
    (BF16, 2, 300, 1, 2, 192, 150, None, 0),
    (BF16, 2, 300, 2, 2, 7, 60, None, 0),       # by element
    (F32, 2, 300, 2, 2, 128, 128, None, 0),
    (F32, 2, 300, 1, 3, 72, 91, 0.01, 3),
    (F32, 1, 1500, 1, 2, 64, 64, None, 0),
    (F32, 1, 300, 1, 1, 256, 256, None, 0),
]


@pytest.mark.parametrize("dtype,b,l,hk,h,dk,dv,reset,sliced", PRECISE)
def test_mean_square(dtype, b, l, hk, h, dk, dv, reset, sliced):
    say("lattn precision", dtype, b, l, hk, h, dk, dv, reset, sliced)
    args, extra, normal = make(dtype, b, l, hk, h, dk, dv, 21, True, reset, sliced)
    do, dh = normal(b, l, h, dv), normal(b, h, dk, dv, dtype=F32)
    got, want = run(args, extra, do, dh, dk ** -0.5)
    for n in want:
        e = float(np.sqrt(np.mean((host64(got[n]) - want[n]) ** 2) / np.mean(want[n] ** 2)))
        state = n in ("h_last", "dh0")
        terms = l if state else max(dk, dv) + l
        bar = TWICE if dtype is BF16 and not state else 2.0 ** -23 + 2.0 ** -24 * np.sqrt(6 * terms / 16 / 2)
        say("   %-7s rms err %.3e (bar %.3e)" % (n, e, bar))
        assert e <= bar, (n, e, bar)


@pytest.mark.parametrize("dtype,l,hk,h,dk,dv,reset", [
    (BF16, 2111, 1, 2, 5, 7, 0.001), (F32, 1100, 2, 2, 3, 40, 0.002), (BF16, 1500, 1, 1, 7, 130, None),
    (F32, 1200, 1, 2, 2, 65, 0.002), (BF16, 1400, 1, 2, 130, 6, None), (F32, 900, 1, 1, 1, 1, 0.01)])
def test_single_elements_in_segments(dtype, l, hk, h, dk, dv, reset):
    """Heads of less than 16 bytes, of sequences that are cut."""
    import selective_state_space_85_amd as ss

    say("lattn single elements", dtype, l, hk, h, dk, dv, reset)
    assert ss.lattn_workspace_bytes(1, l, hk, h, dk, dv, dtype) > 0
    args, extra, normal = make(dtype, 1, l, hk, h, dk, dv, 22, True, reset)
    do, dh = normal(1, l, h, dv), normal(1, h, dk, dv, dtype=F32)
    got, want = run(args, extra, do, dh, 0.5)
    for n in want:
        check(n, got[n], want[n], dtype, max(dk, dv) + l + 3, state=n in ("h_last", "dh0"))
