"""The recurrence's series for 1 - a^2 (no GPU): its coefficients, as the kernel's source has them, in
float32 steps against expm1."""
import os
import re

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def coefficients():
    text = open(os.path.join(ROOT, "selective_state_space_85_amd", "csrc", "ss_glr.hip")).read()
    body = text[text.index("void decay_of("):]
    body = body[:body.index("}")]
    first = re.search(r"float p = fmaf\(t, ([-\d.]+)f, ([-\d.]+)f\);", body)
    rest = re.findall(r"p = fmaf\(t, p, ([-\d.]+)f\);", body)
    assert len(rest) == 3 and "t < 0.5f ? t * p" in body
    return [np.float32(v) for v in (*first.groups(), *rest)]


def fma(a, b, c):
    # exact in float64 but for the sum's rounding, 2^-53
    return (a.astype(np.float64) * np.asarray(b, np.float64) + np.float64(c)).astype(np.float32)


def test_bounds():
    c = coefficients()
    rng = np.random.default_rng(0)
    t = np.concatenate([np.exp(rng.uniform(np.log(1e-12), np.log(0.5), 500000)), rng.uniform(1e-6, 0.5, 1000000)])
    t = t.astype(np.float32)
    t = t[t < 0.5]
    x = t.astype(np.float64)
    want = -np.expm1(-x)
    exact = np.polyval([float(v) for v in c], x)
    assert np.abs(exact / (want / x) - 1).max() <= 1.05e-7
    p = fma(t, c[0], c[1])
    for v in c[2:]:
        p = fma(t, p, v)
    assert np.abs(p / (want / x) - 1).max() <= 1.6e-7
    assert np.abs((t * p) / want - 1).max() <= 2.0e-7
