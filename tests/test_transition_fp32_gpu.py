"""The fp32 transition where its products are taken in parts (few row tiles, or few columns,
beside a long K), against the float64 oracle: every tile and layout, one and many
ranges of K, rows of whole 16-byte units or not in either direction."""
import numpy as np
import pytest
import torch

import triangle_biased_attention_b200 as evo
from oracle import transition as T
from tests.test_transition_gpu import FP32, check, make, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,C,F", [
    (2, 752, 3008), (13, 432, 2075), (33, 1000, 64), (66, 1000, 40), (9, 30, 1055), (40, 270, 300),  # 32 rows a tile
    (124, 688, 2683), (411, 602, 2408), (150, 102, 640), (773, 464, 696),                            # 128 x 128
    (2011, 16, 2775), (700, 72, 200), (257, 61, 1000),                                               # 128 x 64
    (130, 128, 512), (300, 100, 97), (1024, 256, 1024),
    (1, 40, 5001), (3, 4200, 24), (70, 5000, 30),                                                    # too long for the few-row form
], ids=str)
def test_matches_oracle(M, C, F, act):
    check(*make(M, C, F, FP32, seed=M + C), act, f"{M} {C} {F} {act}")


@pytest.mark.parametrize("M,C,F", [(57363, 384, 29), (24000, 40, 3001), (20000, 100, 2500)])
def test_many_rows(M, C, F):
    """Many rows beside few features, and more rows than one chunk: forward and dX at sampled
    rows, the weight gradients of stretches of rows (dY is zero elsewhere)."""
    x, wg, wu, wd, dy = make(M, C, F, FP32, seed=M)
    y = evo.transition(x, wg, wu, wd)
    at = torch.cat([torch.arange(0, M, 97), torch.arange(18944 - 20, 18944 + 20), torch.arange(M - 70, M)])
    ref, err = T.forward(x[at], wg, wu, wd, "silu", FP32)
    within(y[at], ref, err, "y")
    for lo, n in ((0, 100), (18944 - 60, 120), (M - 90, 90)):
        some = torch.zeros_like(dy)
        some[lo:lo + n] = dy[lo:lo + n]
        dx, *dw = evo.transition_backward(x, wg, wu, wd, some)
        ref, err = T.backward(x[lo:lo + n], wg, wu, wd, some[lo:lo + n], "silu", FP32)
        for name, g, r, e in zip(("dx", "dw_gate", "dw_up", "dw_down"), (dx[lo:lo + n], *dw), ref, err):
            assert (np.abs(r) > e).mean() > 0.9, name
            within(g, r, e, f"{M} {C} {F} rows {lo} {name}")
        assert (dx[:lo] == 0).all() and (dx[lo + n:] == 0).all()
    assert evo.evo_attn_sync_status() == evo.EVO_OK


@pytest.mark.parametrize("M,C,F", [(124, 100, 400), (20, 256, 1024), (500, 64, 700)])
def test_unaligned_same_bits_streams_and_graph(M, C, F):
    def shifted(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
        buf[1:] = t.flatten()
        return buf[1:].view(t.shape)
    args = make(M, C, F, FP32, seed=3)
    check(*(shifted(t) for t in args), "silu", "unaligned")
    want = [evo.transition(*args[:4]), *evo.transition_backward(*args)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = [evo.transition(*args[:4], stream=side), *evo.transition_backward(*args, stream=side)]
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    bufs = [t.clone() for t in args]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [evo.transition(*bufs[:4]), *evo.transition_backward(*bufs)]
    other = make(M, C, F, FP32, seed=4)
    for case in (other, args):
        for buf, t in zip(bufs, case):
            buf.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, [evo.transition(*case[:4]), *evo.transition_backward(*case)]))
    none, *dw = evo.transition_backward(*args, need_dx=False)
    assert none is None and all(torch.equal(a, b) for a, b in zip(dw, want[2:]))
    assert torch.equal(evo.transition_backward(*args, need_dw=False)[0], want[1])
    out = torch.full((M + 3, C), 5.0, device="cuda")
    evo.transition(*args[:4], out=out[:M])
    assert torch.equal(out[:M], want[0]) and (out[M:] == 5).all()


@pytest.mark.parametrize("M,C,F", [(3, 64, 96), (124, 100, 400), (20, 256, 1024), (7000, 128, 64)])
def test_outputs_that_are_not_16_byte_aligned(M, C, F):
    def hole(*shape):
        return torch.full((int(np.prod(shape)) + 5,), 7.0, device="cuda")[1:]
    x, wg, wu, wd, dy = args = make(M, C, F, FP32, seed=5)
    want = [evo.transition(*args[:4]), *evo.transition_backward(*args)]
    buf = hole(M, C)
    assert torch.equal(evo.transition(*args[:4], out=buf[:M * C].view(M, C)), want[0]) and (buf[M * C:] == 7).all()
    bufs = [hole(*t.shape) for t in want[1:]]
    ws = torch.empty(evo.evo_transition_bwd_workspace_size(M, C, F, evo.EVO_DTYPE_FP32), dtype=torch.uint8, device="cuda")
    st = evo.evo_transition_bwd(*(t.data_ptr() for t in args), *(b.data_ptr() for b in bufs), ws.data_ptr(), ws.numel(), M, C,
                                F, evo.EVO_ACT_SILU, evo.EVO_DTYPE_FP32, None)
    torch.cuda.synchronize()
    assert st == evo.EVO_OK
    for b, t in zip(bufs, want[1:]):
        assert torch.equal(b[:t.numel()].view(t.shape), t) and (b[t.numel():] == 7).all()
