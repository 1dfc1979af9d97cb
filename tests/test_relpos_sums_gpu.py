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
