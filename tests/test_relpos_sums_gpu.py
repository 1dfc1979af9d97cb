"""The order and the depth of the table gradient's sums, and calls of many batches."""
import numpy as np
import pytest
import torch

import triangle_biased_attention_b200 as evo
from oracle import relpos as R
from oracle.transition import _f64, units
from tests.test_relpos_gpu import BF16, DEPTH, DEV, FP16, FP32, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [BF16, FP16, FP32], ids=lambda d: str(d)[6:])
@pytest.mark.parametrize("B,Sq,Sk", [(2, 301, 100), (1, 77, 9), (1, 1001, 56), (3, 40, 1), (1, 333, 1000), (1, 130, 264)])
def test_same_bits_by_table_and_by_search(B, Sq, Sk, dt):
    """Rows of one warp that end at different times, and lanes that search the borders for
    different lengths, change neither the order of the additions nor, with it, a bit: a border too far
    for the distance table sends every pair through the search."""
    _, borders, pq, pk, _, _, pair = make(B, Sq, Sk, 3, 40, dt, seed=Sq)
    far = torch.cat([borders, torch.tensor([2 ** 30], dtype=torch.int32, device=DEV)])
    near = evo.relpos_bias_backward(pair, borders, pq, pk)
    for _ in range(3):
        assert torch.equal(evo.relpos_bias_backward(pair, borders, pq, pk), near)
        searched = evo.relpos_bias_backward(pair, far, pq, pk)
        assert torch.equal(searched[:-1], near) and (searched[-1] == 0).all()
    assert evo.evo_attn_sync_status() == evo.EVO_OK


def far_bucket(H, Sq, Sk, nb):
    """Most pairs in the last bucket, and columns between them that change their bucket with every row."""
    borders = torch.arange(1001 - nb, 1001, dtype=torch.int32, device=DEV)
    pq = (10 * (torch.arange(Sq) % 2)).to(torch.int32).view(1, -1).to(DEV)
    pk = torch.full((1, Sk), -2000, dtype=torch.int32, device=DEV)
    pk[:, ::8] = -995  # from the fifth bucket before the last to the last and back
    # a value whose last bits every sum past 2^15 rounds away in the same direction
    value = 1 + 2.0 ** -9 - 2.0 ** -23
    want = np.zeros(nb + 1)
    moving, steady = len(range(0, Sk, 8)), Sk - len(range(0, Sk, 8))
    for d in (995, 1005):
        want[int((borders.cpu().numpy() <= d).sum())] += value * (Sq // 2) * moving
    want[nb] += value * Sq * steady
    return borders, pq, pk, value, want


def test_sums_of_one_sign_in_a_long_column():
    """As many heads and buckets as fill the SMs, so that a block could take every query
    row: 65536 additions of one sign into a bin, if it did."""
    H, Sq, Sk, nb = 19, 8192, 1024, 2040
    borders, pq, pk, value, want = far_bucket(H, Sq, Sk, nb)
    dpair = torch.full((1, 1, H, Sq, Sk), value, device=DEV)
    got = _f64(evo.relpos_bias_backward(dpair, borders, pq, pk))
    assert evo.evo_attn_sync_status() == evo.EVO_OK
    gamma = DEPTH * 2.0 ** -24 / (1 - DEPTH * 2.0 ** -24)
    assert (np.abs(got - want[:, None]) <= (gamma + 2.0 ** -24) * want[:, None]).all(), \
        float((np.abs(got - want[:, None]) / np.maximum(want[:, None], 1e-300)).max())


@pytest.mark.parametrize("B", [3000, 40000])
def test_sums_over_many_batches(B):
    """One tile a batch: the last sum is as long as there are batches."""
    value = 1 + 2.0 ** -9 - 2.0 ** -23
    borders = torch.tensor([0], dtype=torch.int32, device=DEV)
    pos = torch.zeros(B, 128, dtype=torch.int32, device=DEV)
    dpair = torch.full((B, 1, 1, 128, 128), value, device=DEV)
    got = _f64(evo.relpos_bias_backward(dpair, borders, pos))
    assert evo.evo_attn_sync_status() == evo.EVO_OK
    want = np.array([[0.0], [value * B * 128 * 128]])
    gamma = DEPTH * 2.0 ** -24 / (1 - DEPTH * 2.0 ** -24)
    assert (np.abs(got - want) <= (gamma + 2.0 ** -24) * want).all(), got[1, 0] / want[1, 0] - 1


@pytest.mark.parametrize("B,H,dt,extra", [(20001, 16, FP32, True), (33000, 9, BF16, False), (65535, 3, FP16, True)], ids=str)
def test_more_batches_and_heads_than_a_grid_dimension(B, H, dt, extra):
    """Batches times groups of heads past 65535: each batch with its own positions, chains and base."""
    table, borders, pq, pk, cq, ck, pair = make(B, 2, 3, H, 7, dt, seed=B, chains=extra)
    base = pair if extra else None
    p = evo.relpos_bias(table, borders, pq, pk, cq, ck, base=base)
    assert evo.evo_attn_sync_status() == evo.EVO_OK
    ref, (r, tiny) = R.forward(table, borders, pq, pk, cq, ck, base), units(dt)
    # exact without a base; with one an fp32 sum and a rounding
    err = (r + 2.0 ** -24) * (1 + 2.0 ** -7) * np.abs(ref) + tiny if extra else 0.0
    assert (np.abs(_f64(p) - ref) <= err).all()
