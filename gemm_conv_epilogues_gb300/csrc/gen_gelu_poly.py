"""Generates gelu_poly.h: the polynomial the GELU kernels use for the normal
tail Q(t) = P(Z > t) = 0.5*erfc(t/sqrt 2).

Method (this library's own): log2 Q(t) is smooth on [0, 6], so it is fitted
by least squares in the Chebyshev basis of v = t/3 - 1 (degree 7) and
converted to power-basis coefficients for Horner evaluation in fp32.  Then
Q(t) = 2^P(v) costs one ex2.approx, and GELU(s) = s*Phi(s) with
Phi(s) = 1 - Q(s) for s >= 0 and Q(-s) for s < 0.  Beyond the fit range the
polynomial keeps falling steeply (P(v) < -29 for v >= 1), so t is clamped at
T_CLAMP = 12 rather than 6: for 6 < t <= 12 the exact |s*Q(t)| is below
6e-9 and the extrapolated 2^P is below 1e-9, and for |s| > 12 the clamped
2^P(3) ~ 2^-111 makes s*Q vanish, so every such output rounds to +-0 in fp16
(and GELU(+inf) = +inf) without a separate test for large |s|.

bf16 has the exponents that fp16 lacks: there s*Q(-s) is a number down to
s = -13.5.  Below -6 the kernels that store bf16 take
t*Q(t) = S(1/t^2) * 2^(-t^2/2 * log2 e) / sqrt(2 pi), the scale of Q's asymptotic
series, with S a quadratic fitted on t in [6, 15]; with phi the density,
Q(t) - t*phi(t), the slope of GELU at -t, is t*phi(t)*(S/t^2 - 1).

The script also checks the whole fp32 evaluation, emulated in numpy, against
s*ndtr(s) on every finite fp16 input: the result must stay within 1 fp16 ulp
of the correctly rounded value (the GPU tests allow 2).
Run: python gen_gelu_poly.py  (needs numpy and scipy; writes gelu_poly.h).
"""
import os

import numpy as np
from scipy.special import log_ndtr, ndtr

T_MAX = 6.0
T_CLAMP = 12.0
DEGREE = 7
T_FAR = 15.0       # fp32's and bf16's t*Q(t) is zero from 14.4 on
FAR_SCALE = 32     # the exponent is evaluated 2^32 too high: ex2 flushes what fp32 still holds


def fit():
    t = np.linspace(0.0, T_MAX, 40001)
    g = log_ndtr(-t) / np.log(2.0)
    v = t / (T_MAX / 2.0) - 1.0
    c = np.polynomial.chebyshev.chebfit(v, g, DEGREE)
    return np.polynomial.chebyshev.cheb2poly(c).astype(np.float32)


def fit_far():
    """S(u), u = 1/t^2, at the Chebyshev points of u over t in [T_MAX, T_FAR]; power basis."""
    lo, hi = 1 / T_FAR ** 2, 1 / T_MAX ** 2
    u = (lo + hi) / 2 + (hi - lo) / 2 * np.cos(np.pi * (np.arange(2000) + 0.5) / 2000)
    t = 1 / np.sqrt(u)
    s = np.exp(log_ndtr(-t) + 0.5 * t * t) * t * np.sqrt(2 * np.pi)
    return np.polynomial.Polynomial.fit(u, s, 2, domain=[lo, hi]).convert().coef.astype(np.float32)


def far_fp32(s32, c):
    """(GELU(s), GELU'(s)) for s < -T_MAX, the kernels' arithmetic step by step in fp32 (ex2 and the
    reciprocal taken exact, results below the smallest normal number of ex2 flushed)."""
    f32, f64 = np.float32, np.float64
    fma = lambda a, b, d: (a.astype(f64) * f64(b) + f64(d)).astype(f32)
    t = np.minimum(np.abs(s32), f32(T_FAR))
    t2 = (t * t).astype(f32)
    e = np.exp2(fma(t2, f32(-0.5 / np.log(2)), f32(FAR_SCALE - 0.5 * np.log2(2 * np.pi))).astype(f64))
    e = np.where(e < 2.0 ** -126, 0, e).astype(f32)
    u = (1 / t2.astype(f64)).astype(f32)
    s = fma(fma(np.full_like(u, c[2]), u.astype(f64), c[1]), u.astype(f64), c[0])
    small = f32(2.0 ** -FAR_SCALE)
    return (-(e * s) * small).astype(f32), ((e * t) * fma(s, u.astype(f64), -1) * small).astype(f32)


def gelu_fp32(s32, p):
    """The kernel's arithmetic, step by step in fp32 (each fmaf as one rounding
    of the double-precision a*b+c; ex2 taken exact)."""
    f64 = np.float64
    t = np.minimum(np.abs(s32), np.float32(T_CLAMP))
    v = (t.astype(f64) * f64(np.float32(1.0 / (T_MAX / 2.0))) - 1.0).astype(np.float32)
    acc = np.full_like(v, p[-1])
    for k in range(len(p) - 2, -1, -1):
        acc = (acc.astype(f64) * v.astype(f64) + f64(p[k])).astype(np.float32)
    q = np.exp2(acc.astype(np.float64)).astype(np.float32)
    w = (s32 * q).astype(np.float32)
    return np.maximum((s32 - w).astype(np.float32), w)


def check(p):
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    s16 = bits.view(np.float16)
    s16 = s16[np.isfinite(s16)]
    s = s16.astype(np.float64)
    ref = (s * ndtr(s)).astype(np.float16).view(np.uint16).astype(np.int64)
    got = gelu_fp32(s16.astype(np.float32), p).astype(np.float16).view(np.uint16).astype(np.int64)
    key = lambda u: np.where(u & 0x8000, -(u & 0x7FFF), u & 0x7FFF)
    ulp = np.abs(key(got) - key(ref))
    return int(ulp.max()), float((ulp > 0).mean())


def main():
    p, far = fit(), fit_far()
    worst, frac = check(p)
    assert worst <= 1, worst
    here = os.path.dirname(os.path.abspath(__file__))
    with open(os.path.join(here, "gelu_poly.h"), "w") as f:
        f.write("// Generated by gen_gelu_poly.py: least-squares fit of log2 Q(t), Q the upper\n")
        f.write("// tail of the standard normal, in v = t/3 - 1 for t in [0, 6]; power basis,\n")
        f.write(f"// lowest order first; t is clamped at TF_GELU_TCLAMP.  fp16 check over every finite\n// input: max {worst} ulp, "
                f"{100 * frac:.2f}% of inputs off by one.\n")
        f.write("#pragma once\n")
        f.write(f"#define TF_GELU_TMAX {T_MAX:.1f}f\n")
        f.write(f"#define TF_GELU_TCLAMP {T_CLAMP:.1f}f\n")
        f.write(f"#define TF_GELU_POLY_DEGREE {DEGREE}\n")
        for k, c in enumerate(p):
            f.write(f"#define TF_GELU_C{k} {float(c)!r}f\n")
        f.write("// t*Q(t)*sqrt(2 pi)*exp(t^2/2) in 1/t^2, for t in [TF_GELU_TMAX, TF_GELU_TFAR]\n")
        f.write(f"#define TF_GELU_TFAR {T_FAR:.1f}f\n")
        for k, c in enumerate(far):
            f.write(f"#define TF_GELU_FAR{k} {float(c)!r}f\n")
    print(f"max {worst} ulp, {100 * frac:.2f}% off by one")


if __name__ == "__main__":
    main()
