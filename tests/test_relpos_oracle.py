"""The relative-position oracle and the border helpers against scalar loops,
central differences and the log formula."""
import math

import numpy as np
import pytest
import torch

import triangle_biased_attention_b200 as evo
from oracle import relpos as R


def case(seed, B=2, Sq=5, Sk=7, H=3, chains=True):
    rng = np.random.default_rng(seed)
    borders = np.array([-3, -1, 0, 1, 4])
    pq, pk = rng.integers(-6, 7, (B, Sq)), rng.integers(-6, 7, (B, Sk))
    cq, ck = (rng.integers(0, 2, (B, Sq)), rng.integers(0, 2, (B, Sk))) if chains else (None, None)
    table = rng.standard_normal((len(borders) + 1 + chains, H))
    return table, borders, pq, pk, cq, ck, rng.standard_normal((B, 1, H, Sq, Sk))


@pytest.mark.parametrize("chains", [False, True])
def test_forward_matches_scalar_loops(chains):
    table, borders, pq, pk, cq, ck, base = case(0, chains=chains)
    p = R.forward(table, borders, pq, pk, cq, ck, base)
    for b, _, h, i, j in np.ndindex(p.shape):
        d = pq[b, i] - pk[b, j]
        r = 0
        while r < len(borders) and borders[r] <= d:
            r += 1
        if chains and cq[b, i] != ck[b, j]:
            r = len(borders) + 1
        assert p[b, 0, h, i, j] == table[r, h] + base[b, 0, h, i, j]


def test_backward_matches_central_differences():
    table, borders, pq, pk, cq, ck, dp = case(1)
    grad = R.backward(dp, table.shape[0], borders, pq, pk, cq, ck)
    for at in np.ndindex(table.shape):
        lo, hi = table.copy(), table.copy()
        lo[at] -= 0.5
        hi[at] += 0.5
        diff = ((R.forward(hi, borders, pq, pk, cq, ck) - R.forward(lo, borders, pq, pk, cq, ck)) * dp).sum()
        assert abs(diff - grad[at]) <= 1e-12 * max(1, abs(diff))


def test_clip_borders():
    b = evo.relpos_clip_borders(32)
    assert b.dtype == torch.int32 and b.tolist() == list(range(-32, 33))
    d = np.arange(-100, 101)[None]
    r = R.rows(b, d, np.zeros((1, 1)))[0, :, 0]
    assert np.array_equal(r, np.clip(d[0], -33, 32) + 33)
    assert evo.relpos_clip_borders(0).tolist() == [0]
    with pytest.raises(ValueError):
        evo.relpos_clip_borders(-1)


@pytest.mark.parametrize("num,reach", [(32, 128), (64, 512), (8, 20), (4, 2), (128, 40000), (32, 2 ** 31 - 1)])
def test_log_borders(num, reach):
    b = evo.relpos_log_borders(num, reach).tolist()
    assert b == sorted(set(b)) and len(b) <= num - 2
    pos = [t for t in b if t > 0]
    assert [1 - t for t in reversed(pos)] == [t for t in b if t <= 0]       # symmetric in the sign
    half, single = num // 2, num // 4
    assert pos[:single] == list(range(1, single + 1))
    # a distance away from the borders falls where the log formula puts it
    steps = half - single
    for t in pos[single:]:
        x = math.log(t / single) / math.log(reach / single) * steps
        y = math.log((t - 1) / single) / math.log(reach / single) * steps if t - 1 > 0 else -1
        assert math.floor(x + 1e-9) > math.floor(y - 1e-9) and t <= reach


def test_log_borders_refusals():
    for num, reach in ((3, 100), (5, 100), (2, 100), (32, 8), (32, 2 ** 31)):
        with pytest.raises(ValueError):
            evo.relpos_log_borders(num, reach)
