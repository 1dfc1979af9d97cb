"""Weight gradients that add up over several chunks of rows, seen one stretch of rows
at a time.

The bound of a sum over M rows grows like M, the gradients of random data like
sqrt(M), so a bound over all rows would not see a chunk that is lost or written over.
Here dY is zero but for a few hundred rows: every other row adds exact zeros to each
gradient, and the bound is that of those rows alone."""
import numpy as np
import pytest
import torch

import triangle_biased_attention_b200 as evo
from oracle import transition as T
from tests.test_transition_gpu import BF16, FP16, FP32, make, within

pytestmark = pytest.mark.gpu
WAVE = 148 * 128  # chunks are whole waves of 128-row tiles


def chunk_rows(M, C, F, dt):
    """Rows of a chunk: the workspace stops growing there."""
    code = {BF16: evo.EVO_DTYPE_BF16, FP16: evo.EVO_DTYPE_FP16, FP32: evo.EVO_DTYPE_FP32}[dt]
    full = evo.evo_transition_bwd_workspace_size(M, C, F, code)
    rows = WAVE
    while evo.evo_transition_bwd_workspace_size(rows, C, F, code) < full:
        rows += WAVE
    return rows


@pytest.mark.parametrize("M,C,F,dt", [
    (5 * WAVE + 300, 16, 1200, BF16),   # weight gradients kept on chip, added into their slots
    (5 * WAVE + 100, 17, 1201, FP16),   # the same from copies of odd rows
    (3 * WAVE + 300, 136, 1200, BF16),  # slots of row ranges, added by bulk reductions
    (3 * WAVE + 268, 132, 1201, FP16),  # the same from copies of odd rows
    (2100000, 9, 8, FP16),              # three chunks
    (WAVE + 300, 16, 1200, FP32),
    (2 * WAVE + 77, 136, 1200, FP32),
], ids=str)
def test_every_stretch_of_rows_counts(M, C, F, dt):
    rows = chunk_rows(M, C, F, dt)
    assert rows < M
    x, wg, wu, wd, dy = make(M, C, F, dt, seed=M)
    # the first rows, the last ones of the first chunk, those on both sides of its end, the last ones
    for lo, n in ((0, 150), (rows - 120, 100), (rows - 70, 140), (M - 50, 50)):
        some = torch.zeros_like(dy)
        some[lo:lo + n] = dy[lo:lo + n]
        dx, *dw = evo.transition_backward(x, wg, wu, wd, some)
        assert evo.evo_attn_sync_status() == evo.EVO_OK
        ref, err = T.backward(x[lo:lo + n], wg, wu, wd, some[lo:lo + n], "silu", dt)
        for name, g, r, e in zip(("dx", "dw_gate", "dw_up", "dw_down"), (dx[lo:lo + n], *dw), ref, err):
            # a gradient that lacks these rows would be zero: the bound tells them apart
            assert (np.abs(r) > e).mean() > 0.9, name
            within(g, r, e, f"{M} {C} {F} {dt} rows {lo} {name}")
        assert (dx[:lo] == 0).all() and (dx[lo + n:] == 0).all()
