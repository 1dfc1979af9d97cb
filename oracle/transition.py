"""Float64 oracle for the gated transition and its gradients (test
infrastructure only; shares nothing with the CUDA path).

    G = X Wg^T,  U = X Wu^T,  H = act(G) * U,  Y = H Wd^T
    dH = dY Wd,  dG = dH * U * act'(G),  dU = dH * act(G)
    dX = dG Wg + dU Wu,  dWg = dG^T X,  dWu = dU^T X,  dWd = dY^T H

``forward`` and ``backward`` also return, on request, a bound of the error that
fp32 accumulation and one rounding of each stored value can cause, element by
element (derived below, beside the code).  Pinned in
tests/test_transition_oracle.py by scalar loops and central differences.
"""
from __future__ import annotations

import math

import numpy as np
import torch

# act(g) of the kernels in fp32, relative to |act(g)|: exp with a few ulp more for
# larger |g|, one division; erfc's argument is rounded, and the relative
# sensitivity of erfc(z) to z is about 2 z^2, 100 roundings at |g| = 10.
ACT_REL = 2.0 ** -16
# the tensor cores' order of additions inside one instruction is their own
ORDER = 4.0


def _f64(x) -> np.ndarray:
    if isinstance(x, torch.Tensor):
        return x.detach().cpu().to(torch.float64).numpy()
    return np.asarray(x, dtype=np.float64)


_erf = np.vectorize(math.erf, otypes=[np.float64])
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def act(g: np.ndarray, kind: str):
    """act(g) and act'(g)."""
    g = np.asarray(g, dtype=np.float64)
    if kind == "silu":
        e = np.exp(-np.abs(g))  # never overflows
        s = np.where(g >= 0, 1 / (1 + e), e / (1 + e))
        return g * s, s + g * s * (1 - s)
    if kind == "gelu":
        phi = 0.5 * _erfc(-g / math.sqrt(2)) if g.size else g * 0
        return g * phi, phi + g * np.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    raise ValueError(kind)


def gamma(n: int) -> float:
    """ORDER times the error of an fp32 sum of n products relative to the sum of their sizes."""
    u = 2.0 ** -24
    return ORDER * n * u / (1 - n * u)


def units(dtype):
    """Half a step of the type relative to the value, and half its smallest step."""
    f = torch.finfo(dtype)
    return f.eps / 2, f.smallest_normal * f.eps / 2


def forward(x, wg, wu, wd, kind: str, dtype=None):
    """Y [M, C]; with a dtype, also the error bound of each element."""
    x, wg, wu, wd = map(_f64, (x, wg, wu, wd))
    g, u = x @ wg.T, x @ wu.T
    a, _ = act(g, kind)
    h = a * u
    y = h @ wd.T
    if dtype is None:
        return y
    C, F = x.shape[1], wg.shape[0]
    r, tiny = units(dtype)
    ax = np.abs(x)
    eg, eu = gamma(C) * (ax @ np.abs(wg).T), gamma(C) * (ax @ np.abs(wu).T)
    eh = _err_h(a, u, eg, eu, r, tiny)
    ey = eh @ np.abs(wd).T + gamma(F) * ((np.abs(h) + eh) @ np.abs(wd).T)
    return y, ey + r * (np.abs(y) + ey) + tiny


def _err_a(a, eg):
    # |act'| <= 1.13 for silu and gelu
    return 1.13 * eg + ACT_REL * (np.abs(a) + 1.13 * eg) + 2.0 ** -126


def _err_h(a, u, eg, eu, r, tiny):
    ea = _err_a(a, eg)
    e = (np.abs(u) + eu) * ea + np.abs(a) * eu
    return e + (r + 2.0 ** -23) * (np.abs(a * u) + e) + tiny  # the product and the rounding to the type


def backward(x, wg, wu, wd, dy, kind: str, dtype=None):
    """(dX, dWg, dWu, dWd); with a dtype, also their error bounds."""
    x, wg, wu, wd, dy = map(_f64, (x, wg, wu, wd, dy))
    g, u = x @ wg.T, x @ wu.T
    a, da = act(g, kind)
    h, dh = a * u, dy @ wd
    dg, du = dh * u * da, dh * a
    out = (dg @ wg + du @ wu, dg.T @ x, du.T @ x, dy.T @ h)
    if dtype is None:
        return out
    M, C, F = x.shape[0], x.shape[1], wg.shape[0]
    r, tiny = units(dtype)
    ax, ady, awg, awu, awd = map(np.abs, (x, dy, wg, wu, wd))
    eg, eu, edh = gamma(C) * (ax @ awg.T), gamma(C) * (ax @ awu.T), gamma(C) * (ady @ awd)
    ea = _err_a(a, eg)
    # |act''| <= 0.8; act' is a sum of terms of size up to 1.2
    eda = 0.8 * eg + ACT_REL * 1.2
    eh = _err_h(a, u, eg, eu, r, tiny)
    U, DA, DH, A = np.abs(u) + eu, np.abs(da) + eda, np.abs(dh) + edh, np.abs(a) + ea
    edg = U * DA * edh + DH * DA * eu + DH * U * eda
    edg += (r + 2.0 ** -22) * (np.abs(dg) + edg) + tiny
    edu = A * edh + DH * ea
    edu += (r + 2.0 ** -22) * (np.abs(du) + edu) + tiny
    DG, DU, H = np.abs(dg) + edg, np.abs(du) + edu, np.abs(h) + eh
    errs = [edg @ awg + edu @ awu + gamma(2 * F) * (DG @ awg + DU @ awu),
            edg.T @ ax + gamma(M) * (DG.T @ ax),
            edu.T @ ax + gamma(M) * (DU.T @ ax),
            ady.T @ eh + gamma(M) * (ady.T @ H)]
    return out, tuple(e + r * (np.abs(o) + e) + tiny for o, e in zip(out, errs))
