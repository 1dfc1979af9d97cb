"""A block's operators run one after another, forward and backward, as a model
runs them: relative-position bias -> triangle attention -> transition on the
pair representation, then transition, attention and table gradients.  Every step
is checked against its float64 oracle on the values that the GPU handed it."""
import numpy as np
import pytest
import torch

import oracle
import triangle_biased_attention_b200 as evo
from oracle import relpos as R
from oracle import transition as T
from oracle.transition import _f64, units
from tests.parity import check, check_grads

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32], ids=lambda d: str(d)[6:])
@pytest.mark.parametrize("S", [40, 72])
def test_block_forward_and_backward(S, dt):
    H, D, F = 4, 32, 256
    C = H * D
    gen = torch.Generator().manual_seed(S)
    n = lambda *s, k=1.0: (torch.randn(*s, generator=gen) * k).to(dt).cuda()  # noqa: E731
    q, k, v = n(1, S, S, H, D), n(1, S, S, H, D), n(1, S, S, H, D)
    mask = torch.zeros(1, S, 1, 1, S)
    mask[..., S - 5:] = -1e9 if dt != torch.float16 else float("-inf")
    mask = mask.to(dt).cuda()
    chain = (torch.arange(S) >= S // 2).int()[None].cuda()
    pos = torch.cat([torch.arange(S // 2), torch.arange(S - S // 2)]).int()[None].cuda()
    borders = evo.relpos_clip_borders(8).cuda()
    table, base = n(borders.numel() + 2, H), n(1, 1, H, S, S)
    wg, wu, wd, dy = n(F, C, k=C ** -0.5), n(F, C, k=C ** -0.5), n(C, F, k=F ** -0.5), n(1, S, S, C)

    pair = evo.relpos_bias(table, borders, pos, chain=chain, base=base)
    o, lse = evo.evo_attn(q, k, v, mask, pair)
    x = o.view(1, S, S, C)
    y = evo.transition(x, wg, wu, wd)
    dx, *dw = evo.transition_backward(x, wg, wu, wd, dy)
    grads = evo.evo_attn_backward(q, k, v, mask, pair, o, lse, dx.view_as(o))
    dtable = evo.relpos_bias_backward(grads[4], borders, pos, chain=chain)
    assert evo.evo_attn_sync_status() == evo.EVO_OK

    r, tiny = units(dt)
    ref = R.forward(table, borders, pos, pos, chain, chain, base)
    assert np.all(np.abs(_f64(pair) - ref) <= (r + 2.0 ** -24) * (1 + 2.0 ** -7) * np.abs(ref) + tiny)
    o_ref, lse_ref = oracle.attention(*(t.cpu() for t in (q, k, v, mask, pair)))
    check(o, lse, o_ref, lse_ref, dt, f"block {S} {dt}")
    rows = lambda t: t.reshape(-1, C)  # noqa: E731
    ref, err = T.forward(rows(x), wg, wu, wd, "silu", dt)
    assert np.all(np.abs(_f64(rows(y)) - ref) <= err)
    refs, errs = T.backward(rows(x), wg, wu, wd, rows(dy), "silu", dt)
    for g, ref, err in zip((rows(dx), *dw), refs, errs):
        assert np.all(np.abs(_f64(g) - ref) <= err)
    want = oracle.attention_bwd(*(t.cpu() for t in (q, k, v, mask, pair)), dx.view_as(o).cpu())
    names = ("dq", "dk", "dv", "dmask", "dpair")
    if not isinstance(want, dict):
        want = dict(zip(names, want))
    check_grads({a: g.cpu() for a, g in zip(names, grads)}, want, dt, f"block {S} {dt}")
    args = (table.shape[0], borders, pos, pos, chain, chain)
    ref, size = R.backward(grads[4], *args), R.backward(grads[4].abs(), *args)
    gamma = 4096 * 2.0 ** -24 / (1 - 4096 * 2.0 ** -24)  # a chain of at most 4096 additions
    assert np.all(np.abs(_f64(dtable) - ref) <= gamma * size + r * (np.abs(ref) + gamma * size) + tiny)
