"""The polynomial that takes part of the attention's exponentials, in fp32 as the kernel computes it: its error stays
within the 2^-20 that the bounds on weights are derived from (tests/pooltest.py)."""
import os
import re

import numpy as np

import hierarchical_long_context_b200 as lod

SOURCE = os.path.join(os.path.dirname(lod.__file__), "csrc", "lod_pool_tc.cuh")


def coefficients():
    """The polynomial's coefficients from the highest power down, as the source gives them."""
    body = open(SOURCE).read().split("exp2_fma2(float2 x) {")[1].split("return p;")[0]
    named = {k: float(v) for k, v in re.findall(r"(c\d) = ([-\d.e]+)f", body)}
    first, rest = re.search(r"float2 p = (.*?);", body).group(1), re.findall(r"p = ffma2\(p, f, make_float2\((\w[\w.]*), ", body)
    terms = re.findall(r"make_float2\((\w[\w.]*), ", first) + rest
    return [named[t] if t in named else float(t.rstrip("f")) for t in terms]


def test_the_polynomial_keeps_the_bound_of_the_weights():
    c = coefficients()
    assert c[-1] == 1.0 and len(c) >= 4
    f = np.linspace(-0.5, 0.5, 1_000_001).astype(np.float32)
    p = np.full_like(f, np.float32(c[0]))
    for k in c[1:]:  # (a product of two fp32 values is exact in fp64: one rounding, as an fma)
        p = (p.astype(np.float64) * f + np.float64(np.float32(k))).astype(np.float32)
    rel = np.abs(p / np.exp2(f.astype(np.float64)) - 1)
    assert rel.max() < 2.0 ** -20
