"""Host-side checks (no GPU): shapes whose launches would pass HIP's limit, fewer than 2^32 threads
along a grid's axis, are refused before anything is enqueued, and the largest below it are not."""
import os
import shutil
import sys

import pytest

import test_lm_abi as abi
from test_lm_abi import BF16, F32, TESTS, UNSUPPORTED, _host_lib, addr, lib  # noqa: F401
from test_sanitize import _run

ROOT = os.path.dirname(TESTS)


def glr(b, d, **kw):
    """One row per sequence; strides of the dense operands."""
    return dict(b=b, l=1, d=d, **{**dict(xs=d, rs=d, is_=d), **kw})


def step(d):
    return dict(b=1, d=d, xs=d, rs=d, is_=d)


# entry, arguments, the last ones that fit, the first that do not
LIMITS = [
    # 512 threads per 64 channels, or per 32 where a row stride is odd
    ("glr_fwd", {}, glr((1 << 23) - 1, 2), glr(1 << 23, 2)),
    ("glr_fwd", {}, glr((1 << 22) - 1, 34, xs=35), glr(1 << 22, 34, xs=35)),
    ("glr_fwd", {}, glr(1 << 22, 34), glr(1 << 23, 34)),
    # 256 in the backward; the forward's where the kept states are formed again
    ("glr_bwd", dict(gs=2), glr((1 << 24) - 1, 2), glr(1 << 24, 2)),
    ("glr_bwd", dict(gs=2, ckpt=None), glr((1 << 23) - 1, 2), glr(1 << 23, 2)),
    # one channel per thread where rows are not whole groups of four, else four
    ("glr_step", {}, step((1 << 32) - 257), step((1 << 32) - 255)),
    ("glr_step", {}, step(1 << 32), None),
    # streamed: 256 per 16 features
    ("glu_fwd", dict(m=1, k=1, xs=1), dict(f=(1 << 28) - 16), dict(f=1 << 28)),
    ("glu_fwd", dict(m=1, k=1, xs=1, dt=F32), dict(f=(1 << 28) - 16), dict(f=1 << 28)),
    # tiles: 512 per 256 x 128 features (bf16), 256 per 128 x 64 (fp32)
    ("glu_fwd", dict(k=8, xs=8, f=1 << 17), dict(m=(1 << 21) - (1 << 18)), dict(m=1 << 21)),
    ("glu_fwd", dict(k=4, xs=4, f=1 << 17, dt=F32), dict(m=(1 << 20) - (1 << 17)), dict(m=1 << 20)),
    # gradients: in one pass, their sum's; in tiles
    ("glu_bwd", dict(m=8, f=1, dt=F32, wsb=1 << 40), None, dict(k=1 << 29, xs=1 << 29)),
    ("glu_bwd", dict(k=1 << 17, xs=1 << 17, wsb=1 << 40), None, dict(f=1 << 21)),
    # the loss: 256 per 32 entries streamed; its join: 256 per 16 tokens
    ("xent_fwd", dict(n=1, k=1, xs=1), dict(v=(1 << 29) - 32), dict(v=1 << 29)),
    ("xent_fwd", dict(v=1, k=1, xs=1, wsb=1 << 34), dict(n=(1 << 28) - 16), dict(n=1 << 28)),
    # the lists of targets: 256 per 128 entries
    ("xent_bwd", dict(k=8, xs=8, wsb=1 << 44), None, dict(v=1 << 31)),
]


@pytest.mark.parametrize("case", [i for i, c in enumerate(LIMITS) if c[3]])
def test_beyond_the_limit(lib, case):  # noqa: F811
    fn, kw, _, first = LIMITS[case]
    assert getattr(abi, fn)(lib, **kw, **first) == UNSUPPORTED, (fn, first)


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
@pytest.mark.skipif("SS_SANITIZED_LIB" in os.environ, reason="this is the sanitized run")
def test_within_the_limit(tmp_path):
    """Over stub launchers, with the sanitizers on."""
    code = ("import sys; sys.path[:0] = [%r, %r]\n"
            "import sanitize.abi_plugin\n"
            "import test_lm_abi as abi\n"
            "import test_lm_launch_limits as t\n"
            "from selective_state_space_85_amd import _lm\n"
            "lib = _lm.load()\n"
            "for fn, kw, last, _ in t.LIMITS:\n"
            "    if last:\n"
            "        assert getattr(abi, fn)(lib, **kw, **last) == 0, (fn, last)\n"
            "print('limits ok')\n") % (TESTS, ROOT)
    r = _run([sys.executable, "-c", code], {"SS_SANITIZED_LIB": str(_host_lib(tmp_path))})
    assert r.returncode == 0 and "limits ok" in r.stdout, (r.stdout[-2000:], r.stderr[-3000:])
