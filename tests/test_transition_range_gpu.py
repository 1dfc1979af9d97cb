"""Gates far out on both sides, in every form of the transition, against
closed forms in 64 bits: forward and backward.

Every product has a single term: G and U are two channels of X, Wd copies H to
Y, so G, U and dH are exact and what is left is the activation's own error and
the roundings.  Bounds, relative to each result:
- 16-bit: half a step for H (dG, dU) and for Y (dX), and ACT for the activation.
  ACT: the exponent of e^-|g| is rounded, |g| 2^-24 <= 2^-17; the one of
  e^(-g^2/2), at most 88, five times, 88 * 5 * 2^-24 < 2^-15; two units of the
  special functions and a dozen roundings more: below 2^-14.
- fp32: silu a dozen roundings and the exponential's, 2^-20; gelu the rounding
  of erfc's argument, whose relative effect is g^2 2^-23 or so, twice that.
- an exponential below the smallest normal number counts as 0, which is |g| 2^-126
  or, beyond, all of act(g): at most FLOOR.
"""
import math

import numpy as np
import pytest
import torch

import triangle_biased_attention_b200 as evo
from oracle import transition as T

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
ACT, FLOOR = 2.0 ** -14, 2.0 ** -118

GATES = [-3e38, -1e30, -1e20, -1e15, -1e12, -1e6, -3e4, -1000.0, -200.0, -100.0, -90.0, -88.5, -88.0, -87.0, -80.0, -60.0,
         -45.0, -43.5, -42.0, -41.5, -41.0, -30.0, -20.0, -13.0, -10.0, -8.0, -6.0, -5.0, -4.0, -3.0, -1.0, -0.25, -1e-20,
         -0.0, 1e-20, 0.5, 1.0, 4.0, 10.0, 20.0, 41.0, 43.5, 90.0, 1000.0, 3e4]
UPS = [1.0, -3.0, 2.0 ** -10, 1000.0]
FAR_UPS = [1e20, -1e30]  # for gates below -200, whose act is 0: g u overflows, act(g) u does not


def rows(dt, many=0):
    """(gate, up) pairs whose act(gate) up the type holds."""
    lim = torch.finfo(dt).max
    pairs = [(g, u) for u in UPS for g in GATES if abs(g) < lim and max(g, 1.0) * abs(u) < lim]
    if dt != FP16:
        pairs += [(g, u) for u in FAR_UPS for g in GATES if g <= -200.0]
    pairs *= max(1, -(-many // len(pairs)))
    return torch.tensor(pairs, dtype=torch.float64).to(dt).double()


def inputs(pairs, C, F, dt):
    M = pairs.shape[0]
    x, wg, wu, wd = torch.zeros(M, C), torch.zeros(F, C), torch.zeros(F, C), torch.zeros(C, F)
    x[:, 0], x[:, 1] = pairs[:, 0], pairs[:, 1]
    wg[:, 0], wu[:, 1] = 1.0, 1.0
    n = min(C, F)
    wd[torch.arange(n), torch.arange(n)] = 1.0
    return [t.to(dt).cuda() for t in (x, wg, wu, wd)]


def bounds(g, u, d, act, dt):
    """act(g) u, d act(g) and d u act'(g), and the error of each."""
    a, da = T.act(g, act)
    r, tiny = T.units(dt)
    rel = np.full_like(g, ACT)
    if dt == FP32:
        rel = np.full_like(g, 2.0 ** -20) if act == "silu" else 2.0 ** -20 + np.minimum(g * g, 256.0) * 2.0 ** -22
    # the terms of act': p + a (1 - p), where 1 - p carries half a step of 1; Phi + g phi
    if act == "silu":
        e = np.exp(-np.abs(g))
        p = np.where(g >= 0, 1 / (1 + e), e / (1 + e))
        cancel = np.where(g < 20, np.abs(a) * 2.0 ** -23, np.abs(a) * 2 * e)
        size = p + np.abs(a) * np.where(g >= 0, e / (1 + e), 1 / (1 + e))
    else:
        phi = np.exp(-0.5 * np.minimum(np.abs(g), 100.0) ** 2) / math.sqrt(2 * math.pi)
        cancel = 0.0
        size = np.where(np.abs(g) > 1e-300, a / np.where(g == 0, 1.0, g), 0.5) + np.minimum(np.abs(g), 100.0) * phi
    floor = FLOOR * (1 + np.abs(u)) + 2 * tiny
    two = 2 * r + r * r
    return ((a * u, (two + rel) * (1 + two) * np.abs(a * u) + floor),
            (d * a, (two + rel) * (1 + two) * np.abs(d * a) + floor),
            (d * u * da, np.abs(d * u) * (two * np.abs(da) + (1 + two) * (rel * size + cancel)) + floor))


def within(got, ref, err, g, u, what):
    got = T._f64(got)
    bad = ~(np.abs(got - ref) <= err)
    if bad.any():
        i = int(np.argmax(bad))
        raise AssertionError(f"{what}: g = {g[i]:g}, u = {u[i]:g}: {got[i]:g} instead of {ref[i]:g} +- {err[i]:g} ({bad.sum()} rows)")


FORWARD = [
    # C, F, rows of a call (0: all at once), rows at least: 16-bit forms
    (16, 16, 1, 0), (16, 16, 4, 0), (50, 18, 8, 0),  # one row, up to 4, up to 8 without whole 16-byte units
    (16, 16, 0, 0), (128, 256, 0, 0),                # Y of a tile beside its features, up to 128 channels
    (136, 16, 0, 12000),                             # up to 256
    (264, 24, 0, 0), (100, 397, 0, 0),               # H through memory
]


@pytest.mark.parametrize("dt", [BF16, FP16], ids=lambda d: str(d)[6:])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("form", FORWARD, ids=str)
def test_forward_16_bit(form, act, dt):
    C, F, step, many = form
    pairs = rows(dt, many)
    x, wg, wu, wd = inputs(pairs, C, F, dt)
    step = step or x.shape[0]
    y = torch.cat([evo.transition(x[m:m + step], wg, wu, wd, act=act) for m in range(0, x.shape[0], step)])
    assert evo.evo_attn_sync_status() == evo.EVO_OK
    g, u = pairs[:, 0].numpy(), pairs[:, 1].numpy()
    (h, err), _, _ = bounds(g, u, np.ones_like(g), act, dt)
    for c in (0, 1, min(C, F) - 1):
        within(y[:, c], h, err, g, u, f"{form} {act} {dt} channel {c}")


@pytest.mark.parametrize("dt", [BF16, FP16], ids=lambda d: str(d)[6:])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("C,F", [(16, 16), (128, 200), (136, 16), (100, 397), (300, 100)])
def test_backward_16_bit(C, F, act, dt):
    pairs = rows(dt)
    x, wg, wu, wd = inputs(pairs, C, F, dt)
    g, u = pairs[:, 0].numpy(), pairs[:, 1].numpy()
    # one feature's dH a row, a different one in each
    n = min(C, F)
    at, d = np.arange(len(g)) % n, np.where(np.arange(len(g)) % 2, 2.0, -0.5)
    dy = torch.zeros(len(g), C)
    dy[torch.arange(len(g)), torch.from_numpy(at)] = torch.from_numpy(d).float()
    dx, *dw = evo.transition_backward(x, wg, wu, wd, dy.to(dt).cuda(), act=act)
    assert evo.evo_attn_sync_status() == evo.EVO_OK
    _, (du, edu), (dg, edg) = bounds(g, u, d, act, dt)
    within(dx[:, 0], dg, edg, g, u, f"{C} {F} {act} {dt} dG")
    within(dx[:, 1], du, edu, g, u, f"{C} {F} {act} {dt} dU")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("form", [(16, 16, 1, 0), (16, 16, 8, 0), (50, 18, 0, 0), (130, 70, 0, 12000), (136, 24, 0, 12000)], ids=str)
def test_forward_fp32(form, act):
    C, F, step, many = form
    pairs = rows(FP32, many)
    x, wg, wu, wd = inputs(pairs, C, F, FP32)
    step = step or x.shape[0]
    y = torch.cat([evo.transition(x[m:m + step], wg, wu, wd, act=act) for m in range(0, x.shape[0], step)])
    assert evo.evo_attn_sync_status() == evo.EVO_OK
    g, u = pairs[:, 0].numpy(), pairs[:, 1].numpy()
    (h, err), _, _ = bounds(g, u, np.ones_like(g), act, FP32)
    for c in (0, 1, min(C, F) - 1):
        within(y[:, c], h, err, g, u, f"{form} {act} channel {c}")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("C,F,many", [(16, 16, 0), (50, 18, 0), (136, 24, 12000)])
def test_backward_fp32(C, F, many, act):
    pairs = rows(FP32, many)
    x, wg, wu, wd = inputs(pairs, C, F, FP32)
    g, u = pairs[:, 0].numpy(), pairs[:, 1].numpy()
    n = min(C, F)
    at, d = np.arange(len(g)) % n, np.where(np.arange(len(g)) % 2, 2.0, -0.5)
    dy = torch.zeros(len(g), C)
    dy[torch.arange(len(g)), torch.from_numpy(at)] = torch.from_numpy(d).float()
    dx, *dw = evo.transition_backward(x, wg, wu, wd, dy.cuda(), act=act)
    assert evo.evo_attn_sync_status() == evo.EVO_OK
    _, (du, edu), (dg, edg) = bounds(g, u, d, act, FP32)
    within(dx[:, 0], dg, edg, g, u, f"{C} {F} {act} dG")
    within(dx[:, 1], du, edu, g, u, f"{C} {F} {act} dU")


@pytest.mark.parametrize("dt", [BF16, FP16, FP32], ids=lambda d: str(d)[6:])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("C,F", [(16, 16), (136, 24), (300, 100)])
def test_weights_behind_closed_gates_have_no_gradient(C, F, act, dt):
    """Gates from -200 to the end of the type: act and its slope are 0, and so is all that
    hangs on them, also where gate times up overflows."""
    lo, up = (-6e4, 2.0) if dt == FP16 else (-1e30, 1e20)
    x, wg, wu, wd = inputs(torch.tensor([[g, up] for g in np.geomspace(-200.0, lo, 200)]), C, F, dt)
    dy = torch.full_like(x, 0.5)
    y = evo.transition(x, wg, wu, wd, act=act)
    grads = evo.transition_backward(x, wg, wu, wd, dy, act=act)
    assert evo.evo_attn_sync_status() == evo.EVO_OK
    for name, t in zip(("y", "dx", "dw_gate", "dw_up", "dw_down"), (y, *grads)):
        assert float(t.double().abs().max()) <= 2.0 ** -100, (name, float(t.double().abs().max()))


@pytest.mark.parametrize("M,C,F,dt", [(70, 16, 16, BF16), (70, 136, 24, BF16), (70, 300, 100, BF16), (1, 16, 16, BF16),
                                      (70, 16, 16, FP32), (7000, 136, 24, FP32)], ids=str)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_a_sum_past_the_range_is_a_closed_gate(M, C, F, dt, act):
    """G = -6e38, which fp32 does not hold: act's limit, not 0 times infinity."""
    x, wg, wu, wd = inputs(torch.tensor([[-3e38, 1.0]] * M), C, F, dt)
    x[:, 2] = x[:, 0]
    wg[:, 2] = 1.0
    y = evo.transition(x, wg, wu, wd, act=act)
    grads = evo.transition_backward(x, wg, wu, wd, torch.ones_like(x), act=act)
    assert evo.evo_attn_sync_status() == evo.EVO_OK
    assert all((t == 0).all() for t in (y, *grads))


@pytest.mark.parametrize("M,C,F,dt", [(70, 16, 16, BF16), (70, 136, 24, BF16), (70, 300, 100, BF16), (1, 16, 16, BF16),
                                      (70, 16, 16, FP32), (7000, 136, 24, FP32)], ids=str)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_a_sum_past_the_range_is_an_open_gate(M, C, F, dt, act):
    """G = 6e38: act is infinite however small U is, and its slope is 1."""
    x, wg, wu, wd = inputs(torch.tensor([[2.0, 0.5]] * M), C, F, dt)
    x[:, 2] = 2.0
    wg[0, 0], wg[0, 2], wg[1:] = 1.5e38, 1.5e38, 0.0
    y = evo.transition(x, wg, wu, wd, act=act)
    dy = torch.zeros_like(x)
    dy[:, 0] = 0.25
    _, dwg, _, _ = evo.transition_backward(x, wg, wu, wd, dy, act=act)
    assert evo.evo_attn_sync_status() == evo.EVO_OK
    assert (y[:, 0] == float("inf")).all()
    # dWg[0, 0] = sum of dH U X = 0.25 * 0.5 * 2, exact in fp32 up to 2^22 rows
    want = torch.tensor(0.25 * M).to(dt)
    assert float(dwg[0, 0]) == float(want) and float(dwg[0, 2]) == float(want)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,C,F,dt", [(70, 64, 96, BF16), (300, 136, 200, FP16), (65, 50, 70, BF16), (70, 64, 96, FP32),
                                      (5000, 64, 96, FP32)], ids=str)
def test_nan_stays_in_its_row_and_its_feature(M, C, F, dt, act):
    gen = torch.Generator().manual_seed(M)
    x, wg, wu, wd, dy = ((torch.randn(*s, generator=gen) * k).to(dt).cuda() for s, k in
                         (((M, C), 1), ((F, C), C ** -0.5), ((F, C), C ** -0.5), ((C, F), F ** -0.5), ((M, C), 1)))
    clean = evo.transition_backward(x, wg, wu, wd, dy, act=act)
    bad = x.clone()
    bad[M // 2, 3] = float("nan")
    dx, *dw = evo.transition_backward(bad, wg, wu, wd, dy, act=act)
    rest = torch.arange(M) != M // 2
    assert torch.isnan(dx[M // 2]).all() and torch.equal(dx[rest], clean[0][rest])
    assert all(torch.isnan(w).all() for w in dw)
    # a gate weight: its own feature's rows and column of the gradients, none beside it
    bad = wg.clone()
    bad[33, 2] = float("nan")
    assert torch.isnan(evo.transition(x, bad, wu, wd, act=act)).all()
    dx, *dw = evo.transition_backward(x, bad, wu, wd, dy, act=act)
    assert evo.evo_attn_sync_status() == evo.EVO_OK
    rest = torch.arange(F) != 33
    assert torch.isnan(dx).all()
    for w in (dw[0], dw[1], dw[2].T):
        assert torch.isnan(w[33]).all() and torch.isfinite(w[rest]).all()
