"""The two polynomials behind a = 2^l and p = 1 - a of the gated linear recurrence, taken from its source and evaluated step by
step in fp32 on the CPU, against 64 bits: how far they are off, and that they are not off in one direction."""
from __future__ import annotations

import os
import re

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "state_space_sequence_amd", "csrc", "m3_recurrence.hip")
F = np.float32
U = 2.0 ** -24


def coefficients(name):
    """The constants of a function, from the highest power down."""
    with open(SOURCE) as f:
        body = re.search(r"void %s\(float l, float &a, float &p\) \{(.*?)\n\}" % name, f.read(), re.S).group(1)
    return [F(float.fromhex(c)) for c in re.findall(r"-?0x[0-9a-f.]+p[-+]\d+(?=f)", body)]


def fma(a, b, c):
    """a b + c, rounded to 53 bits and then to 24: the product of two fp32 numbers is whole in 64 bits."""
    return (np.asarray(a, np.float64) * b + c).astype(F)


def horner(c, x):
    v = fma(x, c[0], c[1])
    for k in c[2:]:
        v = fma(v, x, k)
    return v


def decay(l):
    n = np.rint(l)
    f = l - n
    z = np.exp2(n.astype(np.float64)).astype(F)
    e = horner(coefficients("decay"), f) * f
    return fma(z, e, z), fma(-z, e, F(1) - z)


def mild_decay(l):
    p = l * horner(coefficients("mild_decay"), l)
    return F(1) - p, p


@pytest.mark.parametrize("how,lo,hi,off_a,off_p", [
    (decay, -0.5, 0.0, 1.7, 2.2), (decay, -1.5, -0.5, 1.7, 2.2), (decay, -126.0, -1.5, 1.7, 1.1), (decay, -1e-3, 0.0, 0.51, 1.9),
    (decay, -1e-6, -1e-30, 0.51, 1.9), (mild_decay, -0.5, 0.0, 1.6, 2.2), (mild_decay, -1.5, -0.5, 3.8, 2.2),
    (mild_decay, -1e-3, 0.0, 0.51, 1.9), (mild_decay, -1e-6, -1e-30, 0.51, 1.9)])
def test_how_far_they_are_off(how, lo, hi, off_a, off_p):
    """In units of 2^-24 of the value. Half of one is a rounding: p has that of the polynomial's last step, of its product (with l or f,
    where it is not small beside 1) and those of the steps before, which count less and less; a has that of its sum, and with one
    polynomial for all of -1.5 .. 0 also p's, which is up to 1.8 times its size."""
    rng = np.random.default_rng(3)
    l = rng.uniform(lo, hi, 1_000_000).astype(F)
    l = l[l < 0]
    a, p = how(l)
    la = np.log(2.0) * l.astype(np.float64)
    ra, rp = a / np.exp(la) - 1, p / -np.expm1(la) - 1
    print("  a %.2f, on average %.3f; p %.2f, %.3f" % (abs(ra).max() / U, ra.mean() / U, abs(rp).max() / U, rp.mean() / U))
    assert abs(ra).max() <= off_a * U and abs(rp).max() <= off_p * U
    # a state of slow decay sums hundreds of steps: what all are off by on average stays a tenth of 2^-24
    assert abs(ra.mean()) <= 0.12 * U and abs(rp.mean()) <= 0.12 * U
