"""The transition oracle against scalar loops, closed forms, central differences
and float64 autograd."""
import math

import numpy as np
import pytest
import torch

from oracle import transition as T


def inputs(M, C, F, seed):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((M, C)), rng.standard_normal((F, C)), rng.standard_normal((F, C)),
            rng.standard_normal((C, F)), rng.standard_normal((M, C)))


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_forward_matches_scalar_loops(kind):
    x, wg, wu, wd, _ = inputs(3, 4, 5, 0)
    y = np.zeros((3, 4))
    for m in range(3):
        for f in range(5):
            g = sum(x[m, c] * wg[f, c] for c in range(4))
            u = sum(x[m, c] * wu[f, c] for c in range(4))
            a = g / (1 + math.exp(-g)) if kind == "silu" else g * 0.5 * (1 + math.erf(g / math.sqrt(2)))
            for c in range(4):
                y[m, c] += a * u * wd[c, f]
    assert np.allclose(T.forward(x, wg, wu, wd, kind), y, rtol=1e-13, atol=1e-13)


def test_activation_closed_forms():
    a, da = T.act(np.array([0.0, 800.0, -800.0]), "silu")
    assert np.allclose(a, [0, 800, 0], atol=1e-300) and np.allclose(da, [0.5, 1, 0], atol=1e-300)
    a, da = T.act(np.array([0.0, 40.0, -40.0]), "gelu")
    assert np.allclose(a, [0, 40, 0], atol=1e-300) and np.allclose(da, [0.5, 1, 0], atol=1e-300)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_backward_matches_central_differences(kind):
    arrays = inputs(3, 4, 5, 1)
    x, wg, wu, wd, dy = arrays
    grads = T.backward(x, wg, wu, wd, dy, kind)
    for n in range(4):
        for at in np.ndindex(arrays[n].shape):
            lo, hi = [a.copy() for a in arrays[:4]], [a.copy() for a in arrays[:4]]
            lo[n][at] -= 1e-5
            hi[n][at] += 1e-5
            diff = ((T.forward(*hi, kind) - T.forward(*lo, kind)) * dy).sum() / 2e-5
            assert abs(diff - grads[n][at]) <= 1e-7 * max(1, abs(diff)), (n, at)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_backward_matches_autograd(kind):
    x, wg, wu, wd, dy = inputs(7, 6, 9, 2)
    ts = [torch.tensor(a, requires_grad=True) for a in (x, wg, wu, wd)]
    g = ts[0] @ ts[1].T
    a = torch.nn.functional.silu(g) if kind == "silu" else torch.nn.functional.gelu(g)
    ((a * (ts[0] @ ts[2].T)) @ ts[3].T).backward(torch.tensor(dy))
    for got, t in zip(T.backward(x, wg, wu, wd, dy, kind), ts):
        assert np.allclose(got, t.grad.numpy(), rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
def test_error_bounds_hold_for_a_rounded_evaluation(dtype):
    """An evaluation in fp32 with H, dG and dU rounded to the type stays inside the
    bounds, and a misplaced one does not."""
    rng = np.random.default_rng(3)
    M, C, F = 40, 24, 56
    mk = lambda *s, k=1.0: torch.tensor(rng.standard_normal(s) * k).to(dtype)  # noqa: E731
    x, wg, wu, wd, dy = mk(M, C), mk(F, C, k=C ** -0.5), mk(F, C, k=C ** -0.5), mk(C, F, k=F ** -0.5), mk(M, C)
    y, ey = T.forward(x, wg, wu, wd, "silu", dtype)
    f = [t.float() for t in (x, wg, wu, wd, dy)]
    rd = lambda t: t.to(dtype).float()  # noqa: E731
    g, u, dh = f[0] @ f[1].T, f[0] @ f[2].T, f[4] @ f[3]
    s = torch.sigmoid(g)
    h = rd(g * s * u)
    assert (np.abs(T._f64(rd(h @ f[3].T)) - y) <= ey).all()
    dg, du = rd(dh * u * (s + g * s * (1 - s))), rd(dh * g * s)
    ref, err = T.backward(x, wg, wu, wd, dy, "silu", dtype)
    got = (dg @ f[1] + du @ f[2], dg.T @ f[0], du.T @ f[0], f[4].T @ h)
    for a, r, e in zip(got, ref, err):
        assert (np.abs(T._f64(rd(a)) - r) <= e).all()
        assert (np.abs(np.roll(r, 1, 0) - r) > e).mean() > 0.5
