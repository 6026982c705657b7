"""Host-side checks (no GPU): linear attention and the norms of its queries and keys take every size whose
launches stay below HIP's limit, fewer than 2^32 threads along a grid's axis, and refuse the next one."""
import os
import shutil
import sys

import pytest

import test_attn_abi as abi
from test_attn_abi import ROOT, TESTS, UNSUPPORTED, _host_lib, addr, lib  # noqa: F401
from test_sanitize import _run


def heads(b, dk=1, dv=1):
    """One row of one head in each of b sequences."""
    return dict(b=b, h=1, hk=1, dk=dk, dv=dv, qs=dk, ks=dk, vs=dv)


def walks(b, dk=1, dv=1):
    return dict(heads(b, dk, dv), l=1)


def back(b, dk=1, dv=1):
    return dict(walks(b, dk, dv), dos=dv)


# operands of up to 2^38 bytes, far apart
FAR = {"qknorm_fwd": dict(zip("q k wq wk pos inv qo ko".split(), (addr(16 * i) for i in range(8)))),
       "qknorm_bwd": dict(zip("q k wq wk pos inv dqo dko dq dk dwq dwk ws".split(), (addr(16 * i) for i in range(13))))}


def tokens(n, width=1, half=0):
    return dict(n=n, hq=1, hk=1, w=width, half=half, qs=width, ks=width)


# entry, the last arguments that fit, the first that do not
LIMITS = [
    # whole eights of workgroups: 128 threads up to 64 columns of v, 256 above, and two slices above 128
    ("lattn_fwd", walks((1 << 25) - 8), walks((1 << 25) - 7)),
    ("lattn_fwd", walks((1 << 24) - 8, 1, 128), walks((1 << 24) - 7, 1, 128)),
    ("lattn_fwd", walks((1 << 23) - 4, 1, 129), walks((1 << 23) - 3, 1, 129)),
    # the gradients' three walks in one launch; dv's and then the two others in two
    ("lattn_bwd", back(11184808), back(11184809)),
    ("lattn_bwd", back((1 << 24) - 8, 64, 65), back((1 << 24) - 7, 64, 65)),
    ("lattn_bwd", back((1 << 23) - 8, 65, 64), back((1 << 23) - 7, 65, 64)),
    # 256 threads for each 128 columns
    ("lattn_step", heads((1 << 24) - 1), heads(1 << 24)),
    ("lattn_step", heads((1 << 24) - 1, 1, 128), heads(1 << 24, 1, 128)),
    ("lattn_step", heads((1 << 23) - 1, 1, 129), heads(1 << 23, 1, 129)),
    # 256 threads for each tile of tokens: 16, or 1024 angles
    *[(fn, tokens(((1 << 24) - 1) * tile, w, half), tokens(((1 << 24) - 1) * tile + 1, w, half))
      for fn in ("qknorm_fwd", "qknorm_bwd") for w, half, tile in ((1, 0, 16), (128, 64, 16), (256, 100, 10), (512, 256, 4))],
]


def call(lib, fn, kw):  # noqa: F811
    return getattr(abi, fn)(lib, **FAR.get(fn, {}), **kw)


@pytest.mark.parametrize("case", range(len(LIMITS)))
def test_beyond_the_limit(lib, case):  # noqa: F811
    fn, _, first = LIMITS[case]
    assert call(lib, fn, first) == UNSUPPORTED, (fn, first)


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
@pytest.mark.skipif("SS_SANITIZED_LIB" in os.environ, reason="this is the sanitized run")
def test_within_the_limit(tmp_path):
    """Over stub launchers, with the sanitizers on."""
    code = ("import sys; sys.path[:0] = [%r, %r]\n"
            "import sanitize.abi_plugin\n"
            "import test_attn_launch_limits as t\n"
            "from selective_state_space_85_amd import _attn\n"
            "lib = _attn.load()\n"
            "for fn, last, _ in t.LIMITS:\n"
            "    assert t.call(lib, fn, last) == 0, (fn, last)\n"
            "print('limits ok')\n") % (TESTS, ROOT)
    r = _run([sys.executable, "-c", code], {"SS_SANITIZED_LIB": str(_host_lib(tmp_path))})
    assert r.returncode == 0 and "limits ok" in r.stdout, (r.stdout[-2000:], r.stderr[-3000:])
