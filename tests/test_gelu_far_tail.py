"""The fit that the grouped products take for GELU and its slope far below zero,
pinned on the CPU: the committed coefficients, evaluated as the kernels do in fp32,
keep their relative accuracy down to the smallest bf16."""
import os
import re
import sys

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "gemm_conv_epilogues_gb300", "csrc")


def test_far_tail_keeps_its_relative_accuracy():
    special = pytest.importorskip("scipy.special")
    sys.path.insert(0, CSRC)
    try:
        import gen_gelu_poly as gen
    finally:
        sys.path.remove(CSRC)
    text = open(os.path.join(CSRC, "gelu_poly.h")).read()
    c = np.array([float(re.search(rf"#define TF_GELU_FAR{k} (\S+)f\n", text).group(1)) for k in range(3)], np.float32)
    assert f"#define TF_GELU_TFAR {gen.T_FAR:.1f}f" in text
    s = -np.linspace(6, 20, 200001).astype(np.float32)
    s64 = s.astype(np.float64)
    y, slope = (v.astype(np.float64) for v in gen.far_fp32(s, c))
    want = s64 * special.ndtr(s64)
    phi = np.exp(-0.5 * s64 * s64) / np.sqrt(2 * np.pi)
    want_slope = special.ndtr(s64) + s64 * phi
    # an exponent of up to 150, rounded three times: 150 * 3 * 2^-24 * ln 2 = 1.9e-5; the fit 4.2e-6; half of the smallest bf16
    for got, w in ((y, want), (slope, want_slope)):
        assert np.all(np.abs(got - w) <= 2.4e-5 * np.abs(w) + 2.0 ** -134)
    assert gen.far_fp32(np.float32([-np.inf]), c)[0] == 0
