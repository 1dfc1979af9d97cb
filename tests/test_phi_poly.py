"""The polynomial behind the 16-bit GELU: its error relative to the normal
distribution's lower tail, evaluated in fp32 as the kernels do."""
import math
import os
import re

import numpy as np

import triangle_biased_attention_b200 as evo

SOURCE = os.path.join(os.path.dirname(evo.__file__), "csrc", "transition_sm100.cuh")


def constants():
    with open(SOURCE) as f:
        found = dict(re.findall(r"constexpr float kPhi(T|C\d) = (-?[\d.]+)f;", f.read()))
    return np.float32(found["T"]), [np.float32(found[f"C{k}"]) for k in range(7)]


def fma(a, b, c):
    return (np.asarray(a, np.float64) * np.asarray(b, np.float64) + np.float64(c)).astype(np.float32)


def test_relative_error_of_the_lower_tail():
    T, C = constants()
    g = np.linspace(0, 13.3, 20001, dtype=np.float32)
    t = (1 / fma(g, T, np.float32(1))).astype(np.float32)
    p = np.full_like(t, C[6])
    for c in reversed(C[:6]):
        p = fma(p, t, c)
    p = (p * t).astype(np.float64)
    want = np.array([0.5 * math.erfc(v / math.sqrt(2)) * math.exp(v * v / 2) for v in g.astype(np.float64)])
    # the fit's 6.3e-7, a rounding of each coefficient and of each step of the sum
    assert np.abs(p / want - 1).max() <= 1.2e-6
