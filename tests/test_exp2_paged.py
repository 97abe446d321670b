"""Error of the FMA-pipe exponential of the paged attention (host check): its
float32 steps repeated with the coefficients of the header."""
import os
import re

import numpy as np

HDR = os.path.join(os.path.dirname(__file__), "..", "exact_attention_112_b200", "csrc", "fa_paged_ptx.cuh")


def _fma(a, b, c):
    return (a.astype(np.float64) * b.astype(np.float64) + c.astype(np.float64)).astype(np.float32)


def _exp2(x):
    body = open(HDR).read()
    body = body[body.index("float2 exp2_fma2_quartic(float2 x)"):]
    m = re.search(r"c1 = ([0-9.e+-]+)f, c2 = ([0-9.e+-]+)f, c3 = ([0-9.e+-]+)f, c4 = ([0-9.e+-]+)f", body)
    c1, c2, c3, c4 = (np.float32(float(v)) for v in m.groups())
    x = np.maximum(x.astype(np.float32), np.float32(-126.0))
    j = (x + np.float32(12582912.0)).astype(np.float32)
    n = (j + np.float32(-12582912.0)).astype(np.float32)
    f = _fma(n, np.float32(-1.0), x)
    q = _fma(np.full_like(f, c4), f, np.full_like(f, c3))
    for c in (c2, c1, np.float32(1.0)):
        q = _fma(q, f, np.full_like(f, c))
    return (q.view(np.int32) + (j.view(np.int32) << np.int32(23))).view(np.float32)


def test_relative_error():
    x = np.linspace(-120.0, 8.0, 1_000_001).astype(np.float32)
    rel = _exp2(x).astype(np.float64) / np.exp2(x.astype(np.float64)) - 1.0
    assert np.abs(rel).max() < 3.2e-6           # 2.9e-6 and the float32 steps' 2^-22
    assert abs(rel.mean()) < 5e-7


def test_masked_scores_and_integers():
    assert _exp2(np.array([-np.inf, -1e30], dtype=np.float32)).max() == np.float32(2.0) ** -126
    n = np.arange(-120, 9).astype(np.float32)
    np.testing.assert_array_equal(_exp2(n), np.exp2(n))
