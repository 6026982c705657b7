"""Host-side checks of include/ss_lm.h (no GPU): exports, sizes, argument validation.

Every call here is rejected by host validation before anything is enqueued, so fake (never
dereferenced) device addresses are enough.
"""
import ctypes
import os
import re
import shutil
import subprocess
import sys

import pytest

from selective_state_space_85_amd import _lib, _lm
from test_sanitize import SAN, _run

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TESTS = os.path.join(ROOT, "tests")
HEADER = os.path.join(ROOT, "include", "ss_lm.h")
BAD = ctypes.c_size_t(-1).value

OK, INVALID, UNSUPPORTED, WORKSPACE, HIP = range(5)
F32, BF16 = 0, 1
BASE, GAP = 0x7E0000000000, 1 << 34


def addr(i, off=0):
    return BASE + i * GAP + off


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from selective_state_space_85_amd import build

        build.build()
    return _lm.load()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?\w+\**\s+\**(ss_\w+)\s*\(", text, flags=re.M))
    assert names == set(_lm.EXPORTS), names ^ set(_lm.EXPORTS)
    for name in names:
        assert hasattr(lib, name), name


def glr_fwd(lib, **kw):
    a = dict(x=addr(0), xs=64, r=addr(1), rs=64, i=addr(2), is_=64, decay=addr(3), c=8.0, h0=None, reset=None,
             y=addr(4), h_last=None, ckpt=None, ws=None, wsb=0, b=2, l=100, d=64, dt=BF16)
    a.update(kw)
    return lib.ss_glr_fwd(a["x"], a["xs"], a["r"], a["rs"], a["i"], a["is_"], a["decay"], a["c"], a["h0"], a["reset"],
                          a["y"], a["h_last"], a["ckpt"], a["ws"], a["wsb"], a["b"], a["l"], a["d"], a["dt"], None)


def glr_bwd(lib, **kw):
    a = dict(x=addr(0), xs=64, r=addr(1), rs=64, i=addr(2), is_=64, decay=addr(3), c=8.0, h0=None, reset=None,
             dy=addr(4), dh_last=None, ckpt=addr(5), dx=addr(6), dr=addr(7), di=addr(8), gs=64, ddecay=addr(9),
             dh0=None, ws=addr(10), wsb=1 << 30, b=2, l=100, d=64, dt=BF16)
    a.update(kw)
    return lib.ss_glr_bwd(a["x"], a["xs"], a["r"], a["rs"], a["i"], a["is_"], a["decay"], a["c"], a["h0"], a["reset"],
                          a["dy"], a["dh_last"], a["ckpt"], a["dx"], a["dr"], a["di"], a["gs"], a["ddecay"], a["dh0"],
                          a["ws"], a["wsb"], a["b"], a["l"], a["d"], a["dt"], None)


def glr_step(lib, **kw):
    a = dict(h=addr(0), x=addr(1), xs=64, r=addr(2), rs=64, i=addr(3), is_=64, decay=addr(4), c=8.0, y=addr(5), b=2,
             d=64, dt=BF16)
    a.update(kw)
    return lib.ss_glr_step(a["h"], a["x"], a["xs"], a["r"], a["rs"], a["i"], a["is_"], a["decay"], a["c"], a["y"],
                           a["b"], a["d"], a["dt"], None)


def glu_fwd(lib, **kw):
    a = dict(x=addr(0), xs=64, wg=addr(1), wu=addr(2), h=addr(3), act=0, ws=None, wsb=0, m=100, k=64, f=96, dt=BF16)
    a.update(kw)
    return lib.ss_glu_fwd(a["x"], a["xs"], a["wg"], a["wu"], a["h"], a["act"], a["ws"], a["wsb"], a["m"], a["k"],
                          a["f"], a["dt"], None)


def glu_bwd(lib, **kw):
    a = dict(x=addr(0), xs=64, wg=addr(1), wu=addr(2), dh=addr(3), dx=addr(4), dwg=addr(5), dwu=addr(6), act=0,
             ws=addr(7), wsb=1 << 30, m=100, k=64, f=96, dt=BF16)
    a.update(kw)
    return lib.ss_glu_bwd(a["x"], a["xs"], a["wg"], a["wu"], a["dh"], a["dx"], a["dwg"], a["dwu"], a["act"], a["ws"],
                          a["wsb"], a["m"], a["k"], a["f"], a["dt"], None)


def xent_fwd(lib, **kw):
    a = dict(x=addr(0), xs=64, w=addr(1), t=addr(2), ignore=-100, loss=addr(3), lse=addr(4), ws=addr(5), wsb=1 << 30,
             n=100, k=64, v=1000, dt=BF16)
    a.update(kw)
    return lib.ss_xent_fwd(a["x"], a["xs"], a["w"], a["t"], a["ignore"], a["loss"], a["lse"], a["ws"], a["wsb"], a["n"],
                           a["k"], a["v"], a["dt"], None)


def xent_bwd(lib, **kw):
    a = dict(x=addr(0), xs=64, w=addr(1), t=addr(2), ignore=-100, lse=addr(3), dloss=addr(4), dx=addr(5), dw=addr(6),
             ws=addr(7), wsb=1 << 30, n=100, k=64, v=1000, dt=BF16)
    a.update(kw)
    return lib.ss_xent_bwd(a["x"], a["xs"], a["w"], a["t"], a["ignore"], a["lse"], a["dloss"], a["dx"], a["dw"], a["ws"],
                           a["wsb"], a["n"], a["k"], a["v"], a["dt"], None)


BIG = 1 << 40
REFUSED = [
    # required pointers
    *[(glr_fwd, {n: None}, INVALID) for n in ("x", "r", "i", "decay", "y")],
    *[(glr_bwd, {n: None}, INVALID) for n in ("x", "r", "i", "decay", "dy", "dx", "dr", "di", "ddecay")],
    *[(glr_step, {n: None}, INVALID) for n in ("h", "x", "r", "i", "decay", "y")],
    *[(glu_fwd, {n: None}, INVALID) for n in ("x", "wg", "wu", "h")],
    *[(glu_bwd, {n: None}, INVALID) for n in ("x", "wg", "wu", "dh", "dwg", "dwu")],
    (glu_bwd, dict(dx=None, dwg=None, dwu=None), INVALID),
    *[(xent_fwd, {n: None}, INVALID) for n in ("x", "w", "t", "loss", "lse")],
    *[(xent_bwd, {n: None}, INVALID) for n in ("x", "w", "t", "lse", "dloss")],
    (xent_bwd, dict(dx=None, dw=None), INVALID),
    # sizes
    *[(f, {n: v}, INVALID) for f in (glr_fwd, glr_bwd) for n in ("b", "l", "d") for v in (0, -1)],
    *[(glr_step, {n: 0}, INVALID) for n in ("b", "d")],
    *[(f, {n: 0}, INVALID) for f in (glu_fwd, glu_bwd) for n in ("m", "k", "f")],
    *[(f, {n: 0}, INVALID) for f in (xent_fwd, xent_bwd) for n in ("n", "k", "v")],
    (glr_fwd, dict(b=BIG, l=BIG), INVALID),
    (glu_fwd, dict(m=BIG, k=BIG, xs=BIG), INVALID),
    (xent_fwd, dict(v=BIG, k=BIG, xs=BIG), INVALID),
    (xent_bwd, dict(n=1 << 50, k=1 << 20, xs=1 << 20), INVALID),
    (glr_fwd, dict(b=1 << 40, l=1), UNSUPPORTED),   # a grid of 2^40 workgroups
    (glu_fwd, dict(m=1 << 38, f=1 << 12), UNSUPPORTED),
    # strides
    *[(f, {n: 63}, INVALID) for f in (glr_fwd, glr_bwd, glr_step) for n in ("xs", "rs", "is_")],
    (glr_bwd, dict(gs=63), INVALID),
    (glr_fwd, dict(xs=1 << 62), UNSUPPORTED),
    (glr_fwd, dict(rs=(1 << 20) + 1), UNSUPPORTED),
    (glr_bwd, dict(gs=(1 << 20) + 1), UNSUPPORTED),
    (glu_fwd, dict(xs=63), INVALID),
    (glu_fwd, dict(xs=68), INVALID),   # rows off a 16-byte boundary
    (xent_fwd, dict(xs=68), INVALID),
    # the decay's sharpness
    *[(f, dict(c=c), INVALID) for f in (glr_fwd, glr_bwd, glr_step)
      for c in (0.0, -1.0, float("nan"), float("inf"))],
    # types
    *[(f, dict(dt=7), UNSUPPORTED) for f in (glr_fwd, glr_bwd, glr_step, glu_fwd, glu_bwd, xent_fwd, xent_bwd)],
    (glu_fwd, dict(act=2), UNSUPPORTED),
    (glu_bwd, dict(act=-1), UNSUPPORTED),
    # alignment
    (glr_fwd, dict(x=addr(0, 1)), INVALID),
    (glr_fwd, dict(y=addr(4, 2), dt=F32), INVALID),
    (glr_fwd, dict(ckpt=addr(5, 2)), INVALID),
    (glr_bwd, dict(ddecay=addr(9, 2)), INVALID),
    (glr_step, dict(h=addr(0, 2)), INVALID),
    (glu_fwd, dict(wg=addr(1, 8)), INVALID),
    (glu_fwd, dict(x=addr(0, 2)), INVALID),
    (glu_fwd, dict(x=addr(0, 1), k=63, ws=addr(7), wsb=1 << 30), INVALID),
    (glu_bwd, dict(dh=addr(3, 1)), INVALID),
    (xent_fwd, dict(t=addr(2, 4)), INVALID),
    (xent_fwd, dict(w=addr(1, 4)), INVALID),
    (xent_bwd, dict(dloss=addr(4, 1)), INVALID),
    # overlaps
    (glr_fwd, dict(y=addr(0)), INVALID),
    (glr_fwd, dict(h_last=addr(4)), INVALID),
    (glr_fwd, dict(h0=addr(6), h_last=addr(6, 4)), INVALID),
    (glr_fwd, dict(ckpt=addr(3)), INVALID),
    (glr_bwd, dict(dx=addr(4)), INVALID),
    (glr_bwd, dict(dr=addr(6, 2)), INVALID),
    (glr_bwd, dict(dr=addr(6, 126), gs=192), INVALID),   # slices of one tensor that share a column
    (glr_bwd, dict(dr=addr(6, 300), gs=192), INVALID),
    (glr_bwd, dict(dh0=addr(9)), INVALID),
    (glr_step, dict(y=addr(0)), INVALID),
    (glr_step, dict(y=addr(2)), INVALID),
    (glu_fwd, dict(h=addr(1)), INVALID),
    (glu_bwd, dict(dwu=addr(5)), INVALID),
    (glu_bwd, dict(dx=addr(0)), INVALID),
    (xent_fwd, dict(lse=addr(3)), INVALID),
    (xent_bwd, dict(dw=addr(1)), INVALID),
    # workspaces
    (glr_fwd, dict(b=1, l=8192), WORKSPACE),
    (glr_fwd, dict(b=1, l=8192, ws=addr(9, 8), wsb=1 << 30), INVALID),
    (glr_fwd, dict(b=1, l=8192, ws=addr(0), wsb=1 << 30), INVALID),
    (glr_bwd, dict(ws=None), WORKSPACE),
    (glr_bwd, dict(wsb=255), WORKSPACE),
    (glr_bwd, dict(ws=addr(6)), INVALID),
    (glu_fwd, dict(k=63), WORKSPACE),  # 100 tokens: in tiles, from padded copies
    (glu_bwd, dict(ws=None), WORKSPACE),
    (glu_bwd, dict(wsb=1000), WORKSPACE),
    (glu_bwd, dict(ws=addr(4)), INVALID),
    (xent_fwd, dict(ws=None), WORKSPACE),
    (xent_fwd, dict(ws=addr(5, 16)), INVALID),
    (xent_bwd, dict(wsb=1000), WORKSPACE),
    (xent_bwd, dict(ws=addr(6)), INVALID),
]


@pytest.mark.parametrize("case", range(len(REFUSED)))
def test_refused_on_the_host(lib, case):
    fn, kw, want = REFUSED[case]
    assert fn(lib, **kw) == want, (fn.__name__, kw)


def test_sizes(lib):
    assert lib.ss_glr_ckpt_bytes(2, 65, 10) == 3 * 2 * 10 * 4
    assert lib.ss_glr_ckpt_bytes(0, 1, 1) == BAD
    assert lib.ss_glr_workspace_bytes(8, 256, 5120) == 0, "one tile of rows"
    assert lib.ss_glr_workspace_bytes(1, 1, 1) == 0
    assert lib.ss_glr_workspace_bytes(1, 131072, 2048) > 0
    for q in (0, 1):
        assert lib.ss_glr_bwd_workspace_bytes(1, 0, 1, q) == BAD
    assert (lib.ss_glr_bwd_workspace_bytes(2, 1000, 96, 0) - lib.ss_glr_bwd_workspace_bytes(2, 1000, 96, 1)
            >= lib.ss_glr_ckpt_bytes(2, 1000, 96))
    assert lib.ss_glu_workspace_bytes(100, 64, 96, BF16) == 0
    assert lib.ss_glu_workspace_bytes(100, 63, 96, BF16) >= (100 + 2 * 96) * 64 * 2
    assert lib.ss_glu_workspace_bytes(64, 63, 96, BF16) == 0, "few tokens: the rows are read as they lie"
    assert lib.ss_glu_workspace_bytes(100, 63, 96, 9) == BAD
    assert lib.ss_glu_bwd_workspace_bytes(100, 64, 97, BF16) == 100 * 2 * 104 * 2
    assert lib.ss_xent_workspace_bytes(10, 64, 129, F32) >= 2 * 2 * 10 * 4 + 10 * 4
    assert lib.ss_xent_bwd_workspace_bytes(10, 64, -1, F32) == BAD
    # the logits are taken in pieces: the workspace stays far below their size
    assert lib.ss_xent_bwd_workspace_bytes(1 << 17, 2560, 1 << 17, BF16) < (1 << 34) // 4


def _host_lib(tmp_path):
    """The C ABI's translation units over stub launchers, built with the host compiler under
    AddressSanitizer and UndefinedBehaviorSanitizer."""
    out = tmp_path / "libssscan_lm_san.so"
    csrc = os.path.join(ROOT, "selective_state_space_85_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-fPIC", "-shared"] + SAN +
                   ["-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    os.path.join(csrc, "ss_api.cpp"), os.path.join(csrc, "ss_lm_api.cpp"),
                    os.path.join(TESTS, "sanitize", "launch_stubs.cpp"),
                    os.path.join(TESTS, "sanitize", "lm_launch_stubs.cpp"), "-o", str(out)], check=True)
    return out


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
@pytest.mark.skipif("SS_SANITIZED_LIB" in os.environ, reason="this is the sanitized run")
def test_validation_under_sanitizers(tmp_path):
    r = _run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "sanitize.abi_plugin", "-p", "no:cacheprovider",
              os.path.join(TESTS, "test_lm_abi.py"), "-m", "not gpu"],
             {"SS_SANITIZED_LIB": str(_host_lib(tmp_path)), "PYTHONPATH": TESTS + os.pathsep + ROOT})
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])
    assert " passed" in r.stdout


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
@pytest.mark.skipif("SS_SANITIZED_LIB" in os.environ, reason="this is the sanitized run")
def test_valid_calls_and_the_hip_failure_path(tmp_path):
    """Valid calls pass validation (the stub launchers answer success), and a failing launch
    returns SS_ERR_HIP and leaves its code in ss_last_hip_error."""
    path = str(_host_lib(tmp_path))
    code = ("import sys; sys.path[:0] = [%r, %r]\n"
            "import sanitize.abi_plugin\n"
            "import test_lm_abi as t\n"
            "from selective_state_space_85_amd import _lm\n"
            "lib, want = _lm.load(), int(sys.argv[1])\n"
            "calls = [(t.glr_fwd, {}), (t.glr_fwd, dict(b=1, l=8192, ws=t.addr(9), wsb=1 << 30)),\n"
            "         (t.glr_fwd, dict(h0=t.addr(6), h_last=t.addr(6))), (t.glr_bwd, {}),\n"
            "         (t.glr_bwd, dict(ckpt=None)), (t.glr_bwd, dict(dr=t.addr(6, 128), di=t.addr(6, 256), gs=192)),\n"
            "         (t.glr_step, {}), (t.glu_fwd, {}), (t.glu_fwd, dict(k=63, ws=t.addr(7), wsb=1 << 30)),\n"
            "         (t.glu_bwd, {}), (t.glu_bwd, dict(dx=None)), (t.xent_fwd, {}),\n"
            "         (t.xent_fwd, dict(k=63)), (t.xent_bwd, {}), (t.xent_bwd, dict(dw=None))]\n"
            "for fn, kw in calls:\n"
            "    assert fn(lib, **kw) == want, (fn.__name__, kw)\n"
            "assert lib.ss_last_hip_error() == (17 if want == 4 else 0)\n"
            "print('calls ok')\n") % (TESTS, ROOT)
    for want, extra in ((0, {}), (4, {"SS_STUB_LAUNCH_ERROR": "17"})):
        r = _run([sys.executable, "-c", code, str(want)], {"SS_SANITIZED_LIB": path, **extra})
        assert r.returncode == 0 and "calls ok" in r.stdout, (r.stdout[-2000:], r.stderr[-3000:])
