"""Host-side checks of include/ss_attn.h (no GPU): exports, sizes, argument validation.

Every call here is rejected by host validation before anything is enqueued, so fake (never
dereferenced) device addresses are enough.
"""
import os
import re
import shutil
import subprocess
import sys

import pytest

from selective_state_space_85_amd import _attn, _lib
from test_lm_abi import BAD, BF16, F32, INVALID, UNSUPPORTED, WORKSPACE, addr
from test_sanitize import SAN, _run

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TESTS = os.path.join(ROOT, "tests")
HEADER = os.path.join(ROOT, "include", "ss_attn.h")
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from selective_state_space_85_amd import build

        build.build()
    return _attn.load()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?\w+\**\s+\**(ss_\w+)\s*\(", text, flags=re.M))
    assert names == set(_attn.EXPORTS), names ^ set(_attn.EXPORTS)
    for name in names:
        assert hasattr(lib, name), name


def _call(fn, names, a, kw):
    a = dict(a, **kw)
    return fn(*[a[n] for n in names.split()], None)


def lattn_fwd(lib, **kw):
    return _call(lib.ss_lattn_fwd, "q qs k ks v vs decay scale h0 reset o h_last ws wsb b l hk h dk dv dt",
                 dict(q=addr(0), qs=128, k=addr(1), ks=128, v=addr(2), vs=160, decay=addr(3), scale=0.125, h0=None,
                      reset=None, o=addr(4), h_last=None, ws=None, wsb=0, b=2, l=100, hk=2, h=4, dk=64, dv=40, dt=BF16), kw)


def lattn_bwd(lib, **kw):
    return _call(lib.ss_lattn_bwd,
                 "q qs k ks v vs decay scale h0 reset do dos dh_last dq dk_ dv_ dh0 ws wsb b l hk h dk dv dt",
                 dict(q=addr(0), qs=128, k=addr(1), ks=128, v=addr(2), vs=160, decay=addr(3), scale=0.125, h0=None,
                      reset=None, do=addr(4), dos=160, dh_last=None, dq=addr(5), dk_=addr(6), dv_=addr(7), dh0=None,
                      ws=addr(8), wsb=1 << 33, b=2, l=100, hk=2, h=4, dk=64, dv=40, dt=BF16), kw)


def lattn_step(lib, **kw):
    return _call(lib.ss_lattn_step, "h_ q qs k ks v vs decay scale o b hk h dk dv dt",
                 dict(h_=addr(5), q=addr(0), qs=128, k=addr(1), ks=128, v=addr(2), vs=160, decay=addr(3), scale=0.125,
                      o=addr(4), b=2, hk=2, h=4, dk=64, dv=40, dt=BF16), kw)


def qknorm_fwd(lib, **kw):
    return _call(lib.ss_qknorm_fwd, "q qs k ks wq wk pos inv eps inter qo ko n hq hk w half dt",
                 dict(q=addr(0), qs=256, k=addr(1), ks=128, wq=addr(2), wk=addr(3), pos=addr(4), inv=addr(5), eps=1e-6,
                      inter=0, qo=addr(6), ko=addr(7), n=50, hq=4, hk=2, w=64, half=32, dt=BF16), kw)


def qknorm_bwd(lib, **kw):
    return _call(lib.ss_qknorm_bwd, "q qs k ks wq wk pos inv eps inter dqo dko dq dk dwq dwk ws wsb n hq hk w half dt",
                 dict(q=addr(0), qs=256, k=addr(1), ks=128, wq=addr(2), wk=addr(3), pos=addr(4), inv=addr(5), eps=1e-6,
                      inter=0, dqo=addr(6), dko=addr(7), dq=addr(8), dk=addr(9), dwq=addr(10), dwk=addr(11), ws=addr(12),
                      wsb=1 << 30, n=50, hq=4, hk=2, w=64, half=32, dt=BF16), kw)


def sample(lib, **kw):
    return _call(lib.ss_sample, "x xs u t ta k ka p pa m ma token ws wsb n v dt",
                 dict(x=addr(0), xs=1000, u=addr(1), t=None, ta=1.0, k=None, ka=0, p=None, pa=1.0, m=None, ma=0.0,
                      token=addr(2), ws=None, wsb=0, n=5, v=1000, dt=BF16), kw)


BIG = 1 << 40
REFUSED = [
    # required pointers
    *[(lattn_fwd, {n: None}, INVALID) for n in ("q", "k", "v", "decay", "o")],
    *[(lattn_bwd, {n: None}, INVALID) for n in ("q", "k", "v", "decay", "do", "dq", "dk_", "dv_")],
    *[(lattn_step, {n: None}, INVALID) for n in ("h_", "q", "k", "v", "decay", "o")],
    *[(f, {n: None}, INVALID) for f in (qknorm_fwd, qknorm_bwd) for n in ("q", "k", "wq", "wk", "pos", "inv")],
    *[(qknorm_fwd, {n: None}, INVALID) for n in ("qo", "ko")],
    *[(qknorm_bwd, {n: None}, INVALID) for n in ("dqo", "dko", "dq", "dk", "dwq", "dwk")],
    *[(sample, {n: None}, INVALID) for n in ("x", "u", "token")],
    # sizes
    *[(f, {n: v}, INVALID) for f in (lattn_fwd, lattn_bwd) for n in ("b", "l", "hk", "h", "dk", "dv") for v in (0, -1)],
    *[(lattn_step, {n: 0}, INVALID) for n in ("b", "hk", "h", "dk", "dv")],
    *[(f, dict(hk=3), INVALID) for f in (lattn_fwd, lattn_bwd, lattn_step)],       # 4 heads by 3
    *[(f, dict(hk=8, qs=512, ks=512), INVALID) for f in (lattn_fwd, lattn_bwd, lattn_step)],
    *[(f, dict(dk=257, qs=1024, ks=1024), UNSUPPORTED) for f in (lattn_fwd, lattn_bwd, lattn_step)],
    *[(f, dict(dv=257, vs=2048, dos=2048), UNSUPPORTED) for f in (lattn_bwd,)],
    (lattn_fwd, dict(b=BIG, l=BIG), INVALID),
    (lattn_fwd, dict(b=1 << 36, l=1), UNSUPPORTED),   # a grid of 2^38 workgroups
    (lattn_bwd, dict(b=1 << 36, l=1), UNSUPPORTED),
    (lattn_step, dict(b=1 << 36), UNSUPPORTED),
    *[(f, {n: 0}, INVALID) for f in (qknorm_fwd, qknorm_bwd) for n in ("n", "hq", "hk", "w")],
    *[(f, dict(half=v), INVALID) for f in (qknorm_fwd, qknorm_bwd) for v in (-1, 33)],
    *[(f, dict(w=513, qs=4096, ks=4096), UNSUPPORTED) for f in (qknorm_fwd, qknorm_bwd)],
    *[(f, dict(n=1 << 32), UNSUPPORTED) for f in (qknorm_fwd, qknorm_bwd)],
    *[(f, dict(n=1, w=1, half=0, **{h: (1 << 24) + 1, s: 1 << 26}), UNSUPPORTED) for f in (qknorm_fwd, qknorm_bwd)
      for h, s in (("hq", "qs"), ("hk", "ks"))],
    *[(f, dict(n=BIG, hq=BIG, qs=BIG), INVALID) for f in (qknorm_fwd, qknorm_bwd)],
    *[(sample, {n: v}, INVALID) for n in ("n", "v") for v in (0, -1)],
    (sample, dict(v=(1 << 24) + 1, xs=1 << 25), UNSUPPORTED),
    (sample, dict(n=1 << 32), UNSUPPORTED),
    (sample, dict(xs=1 << 62, n=100), INVALID),
    # strides
    *[(f, {n: 127}, INVALID) for f in (lattn_fwd, lattn_bwd, lattn_step) for n in ("qs", "ks", "vs")],
    (lattn_bwd, dict(dos=159), INVALID),
    *[(f, {n: (1 << 20) + 1}, UNSUPPORTED) for f in (lattn_fwd, lattn_bwd) for n in ("qs", "ks", "vs")],
    (lattn_bwd, dict(dos=1 << 62), UNSUPPORTED),
    (lattn_step, dict(qs=1 << 62), INVALID),
    (lattn_fwd, dict(l=1 << 30), UNSUPPORTED),
    *[(f, dict(qs=255), INVALID) for f in (qknorm_fwd, qknorm_bwd)],
    *[(f, dict(ks=127), INVALID) for f in (qknorm_fwd, qknorm_bwd)],
    (sample, dict(xs=999), INVALID),
    # numbers
    *[(f, dict(scale=s), INVALID) for f in (lattn_fwd, lattn_bwd, lattn_step) for s in (NAN, INF)],
    *[(f, dict(eps=e), INVALID) for f in (qknorm_fwd, qknorm_bwd) for e in (-1e-9, NAN, INF)],
    # types
    *[(f, dict(dt=7), UNSUPPORTED) for f in (lattn_fwd, lattn_bwd, lattn_step, qknorm_fwd, qknorm_bwd, sample)],
    # alignment
    *[(f, dict(q=addr(0, 1)), INVALID) for f in (lattn_fwd, lattn_bwd, lattn_step, qknorm_fwd, qknorm_bwd)],
    *[(f, dict(decay=addr(3, 2)), INVALID) for f in (lattn_fwd, lattn_bwd, lattn_step)],
    (lattn_fwd, dict(o=addr(4, 2), dt=F32), INVALID),
    (lattn_fwd, dict(h0=addr(6, 2)), INVALID),
    (lattn_bwd, dict(dh0=addr(9, 1)), INVALID),
    (lattn_bwd, dict(dk_=addr(6, 1)), INVALID),
    (lattn_step, dict(h_=addr(5, 2)), INVALID),
    *[(f, dict(pos=addr(4, 4)), INVALID) for f in (qknorm_fwd, qknorm_bwd)],
    *[(f, dict(inv=addr(5, 2)), INVALID) for f in (qknorm_fwd, qknorm_bwd)],
    (qknorm_fwd, dict(ko=addr(7, 1)), INVALID),
    (qknorm_bwd, dict(dwk=addr(11, 2)), INVALID),
    (sample, dict(x=addr(0, 1)), INVALID),
    (sample, dict(token=addr(2, 4)), INVALID),
    (sample, dict(p=addr(3, 2)), INVALID),
    # overlaps
    (lattn_fwd, dict(o=addr(2)), INVALID),
    (lattn_fwd, dict(h_last=addr(4)), INVALID),
    (lattn_fwd, dict(h0=addr(6), h_last=addr(6, 4)), INVALID),
    (lattn_fwd, dict(h0=addr(4)), INVALID),
    (lattn_bwd, dict(dq=addr(5), dk_=addr(5, 64)), INVALID),
    (lattn_bwd, dict(dv_=addr(4)), INVALID),
    (lattn_bwd, dict(dh_last=addr(9), dh0=addr(9)), INVALID),
    (lattn_step, dict(o=addr(2)), INVALID),
    (lattn_step, dict(h_=addr(0)), INVALID),
    (qknorm_fwd, dict(qo=addr(0)), INVALID),
    (qknorm_fwd, dict(ko=addr(6, 256)), INVALID),
    (qknorm_bwd, dict(dq=addr(6)), INVALID),
    (qknorm_bwd, dict(dwk=addr(10)), INVALID),
    (sample, dict(token=addr(1)), INVALID),
    # workspaces
    (lattn_fwd, dict(b=1, l=8192), WORKSPACE),
    (lattn_fwd, dict(b=1, l=8192, ws=addr(7), wsb=64), WORKSPACE),
    (lattn_fwd, dict(b=1, l=8192, ws=addr(7, 128), wsb=1 << 33), INVALID),
    (lattn_fwd, dict(b=1, l=8192, ws=addr(4), wsb=1 << 33), INVALID),
    (lattn_bwd, dict(ws=None), WORKSPACE),     # heads that share: sums of their own
    (lattn_bwd, dict(ws=addr(6)), INVALID),
    (qknorm_bwd, dict(ws=None), WORKSPACE),
    (qknorm_bwd, dict(wsb=2 * 50 * 64 * 4 - 1), WORKSPACE),
    (qknorm_bwd, dict(ws=addr(8)), INVALID),
]


@pytest.mark.parametrize("fn,kw,status", REFUSED, ids=lambda v: getattr(v, "__name__", None) or str(v)[:60])
def test_refused(lib, fn, kw, status):
    assert fn(lib, **kw) == status


def test_workspace_sizes(lib):
    # a walk for every CU: nothing is needed; one long sequence is cut, and needs its states between the cuts
    assert lib.ss_lattn_workspace_bytes(8, 2048, 40, 40, 128, 128, BF16) == 0
    n = lib.ss_lattn_workspace_bytes(1, 131072, 16, 16, 128, 128, BF16)
    assert n > 0 and n % (16 * 128 * 128 * 4) < 1 << 20
    # queries and keys that heads share: the backward forms each head's part first
    assert lib.ss_lattn_bwd_workspace_bytes(8, 2048, 40, 40, 128, 128, BF16) == 0
    assert lib.ss_lattn_bwd_workspace_bytes(8, 2048, 20, 40, 128, 128, BF16) == 2 * 8 * 2048 * 40 * 128 * 4
    for args in ((0, 1, 1, 1, 1, 1, F32), (1, 1, 2, 3, 1, 1, F32), (1, 1, 1, 1, 257, 1, F32), (1, 1, 1, 1, 1, 1, 9),
                 (BIG, BIG, 1, 1, 1, 1, F32)):
        assert lib.ss_lattn_workspace_bytes(*args) == BAD
        assert lib.ss_lattn_bwd_workspace_bytes(*args) == BAD
    assert lib.ss_qknorm_bwd_workspace_bytes(50, 4, 2, 64) == 2 * 50 * 64 * 4
    assert lib.ss_qknorm_bwd_workspace_bytes(1 << 20, 4, 2, 64) < 1 << 24
    assert lib.ss_qknorm_bwd_workspace_bytes(0, 4, 2, 64) == BAD
    assert lib.ss_qknorm_bwd_workspace_bytes(1, 1, 1, 513) == BAD
    for args in ((0, 10, F32), (10, 0, F32), (1, 1 << 25, F32), (1, 10, 5)):
        assert lib.ss_sample_workspace_bytes(*args) == BAD


def _host_lib(tmp_path):
    """The C ABI's translation units over stub launchers, built with the host compiler under
    AddressSanitizer and UndefinedBehaviorSanitizer."""
    out = tmp_path / "libssscan_attn_san.so"
    csrc = os.path.join(ROOT, "selective_state_space_85_amd", "csrc")
    units = [os.path.join(csrc, n) for n in ("ss_api.cpp", "ss_lm_api.cpp", "ss_attn_api.cpp")]
    stubs = [os.path.join(TESTS, "sanitize", n + ".cpp") for n in ("launch_stubs", "lm_launch_stubs", "attn_launch_stubs")]
    subprocess.run(["g++", "-std=c++17", "-fPIC", "-shared"] + SAN +
                   ["-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", csrc]
                   + units + stubs + ["-o", str(out)], check=True)
    return out


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
@pytest.mark.skipif("SS_SANITIZED_LIB" in os.environ, reason="this is the sanitized run")
def test_validation_under_sanitizers(tmp_path):
    r = _run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "sanitize.abi_plugin", "-p", "no:cacheprovider",
              os.path.join(TESTS, "test_attn_abi.py"), "-m", "not gpu"],
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
            "import test_attn_abi as t\n"
            "from selective_state_space_85_amd import _attn\n"
            "lib, want = _attn.load(), int(sys.argv[1])\n"
            "a = t.addr\n"
            "calls = [(t.lattn_fwd, {}), (t.lattn_fwd, dict(b=1, l=8192, ws=a(9), wsb=1 << 33)),\n"
            "         (t.lattn_fwd, dict(h0=a(6), h_last=a(6), reset=a(7))), (t.lattn_fwd, dict(q=a(0, 2), dt=t.BF16)),\n"
            "         (t.lattn_fwd, dict(q=a(0), k=a(0), qs=512, ks=512)),\n"
            "         (t.lattn_bwd, {}), (t.lattn_bwd, dict(dh0=a(9), dh_last=a(10), h0=a(11))),\n"
            "         (t.lattn_bwd, dict(b=1, l=8192)), (t.lattn_bwd, dict(hk=4, qs=256, ks=256, dv=64, vs=256, dos=256)),\n"
            "         (t.lattn_step, {}), (t.qknorm_fwd, {}), (t.qknorm_fwd, dict(inv=None, half=0)), (t.qknorm_bwd, {}),\n"
            "         (t.sample, {}), (t.sample, dict(t=a(3), k=a(4), p=a(5), m=a(6)))]\n"
            "for fn, kw in calls:\n"
            "    assert fn(lib, **kw) == want, (fn.__name__, kw)\n"
            "assert lib.ss_last_hip_error() == (17 if want == 4 else 0)\n"
            "print('calls ok')\n") % (TESTS, ROOT)
    for want, extra in ((0, {}), (4, {"SS_STUB_LAUNCH_ERROR": "17"})):
        r = _run([sys.executable, "-c", code, str(want)], {"SS_SANITIZED_LIB": path, **extra})
        assert r.returncode == 0 and "calls ok" in r.stdout, (r.stdout[-2000:], r.stderr[-3000:])
