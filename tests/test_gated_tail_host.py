"""The normal distribution's tail as the gated kernels evaluate it: the coefficients in the source against the
scaled complementary error function in 64 bits, and their evaluation in fp32."""

import os
import re

import numpy as np
from scipy.special import erfcx

import dense_gemm_tuning_amd as dgt

f = np.float32
U24 = 2.0 ** -24


def coefficients():
    path = os.path.join(os.path.dirname(os.path.abspath(dgt.__file__)), "csrc", "gated.hpp")
    with open(path) as src:
        body = src.read().split("Normal normal(float x)")[1].split("return")[0]
    assert "fmaf(0.4f, fabsf(x), 1.0f)" in body and "0.5f * bell * t * q" in body and "-0.72134752f * (x * x)" in body
    first = re.search(r"float q = (-?[\d.]+)f;", body).group(1)
    return [f(c) for c in [first] + re.findall(r"q = fmaf\(q, t, (-?[\d.]+)f\);", body)]


def fma(a, b, c):
    """In 64 bits a product of two fp32 numbers is exact and the sum's rounding far below fp32's."""
    return (np.float64(a) * np.float64(b) + np.float64(c)).astype(f)


X = np.concatenate([np.linspace(0, 60, 300001), np.logspace(-8, 2, 20001)])


def test_the_fit():
    t = 1 / (1 + 0.4 * X)
    q = np.zeros_like(t)
    for c in coefficients():
        q = q * t + np.float64(c)
    assert len(coefficients()) == 10
    assert np.abs(q * t / erfcx(X / np.sqrt(2)) - 1).max() < 1.44e-7


def test_its_evaluation():
    x = X.astype(f)
    t = (1 / np.float64(fma(f(0.4), x, f(1)))).astype(f)
    co = coefficients()
    q = np.full_like(t, co[0])
    for c in co[1:]:
        q = fma(q, t, c)
    assert np.abs(np.float64(t * q) / erfcx(np.float64(x) / np.sqrt(2)) - 1).max() < 4.1e-7


def test_the_exponentials_argument():
    """x*x and the product with log2(e)/2 are each rounded, as that constant is: the exponential is off by x^2/2 times
    the three."""
    x = X[X < 12].astype(f)
    got = np.exp2(np.float64(f(-0.72134752) * (x * x)))
    want = np.exp(-np.float64(x) ** 2 / 2)
    assert (np.abs(got / want - 1) <= 1.01 * np.float64(x) ** 2 * U24 + 1e-15).all()
