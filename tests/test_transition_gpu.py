"""The gated transition on the GPU against the float64 oracle, element by element
within the error that fp32 accumulation and the documented roundings can cause
(oracle/transition.py derives it)."""
import numpy as np
import pytest
import torch

import triangle_biased_attention_b200 as evo
from oracle import transition as T

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def make(M, C, F, dt, seed, dev="cuda:0"):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s, k=1.0: (torch.randn(*s, generator=gen) * k).to(dt).to(dev)  # noqa: E731
    return n(M, C), n(F, C, k=C ** -0.5), n(F, C, k=C ** -0.5), n(C, F, k=F ** -0.5), n(M, C)


def within(got, ref, err, what):
    got = T._f64(got)
    assert got.shape == ref.shape and np.isfinite(got).all(), what
    ratio = float((np.abs(got - ref) / err).max(initial=0))
    print(f"{what}: max err/bound {ratio:.3f}")
    assert ratio <= 1.0, what


def check(x, wg, wu, wd, dy, act, what, stream=None):
    dt = x.dtype
    y = evo.transition(x, wg, wu, wd, act=act, stream=stream)
    grads = evo.transition_backward(x, wg, wu, wd, dy, act=act, stream=stream)
    assert evo.evo_attn_sync_status(None if stream is None else stream.cuda_stream) == evo.EVO_OK
    torch.cuda.synchronize()
    ref, err = T.forward(x, wg, wu, wd, act, dt)
    within(y, ref, err, f"{what} y")
    ref, err = T.backward(x, wg, wu, wd, dy, act, dt)
    for name, g, r, e in zip(("dx", "dw_gate", "dw_up", "dw_down"), grads, ref, err):
        within(g, r, e, f"{what} {name}")


SHAPES = [
    # M, C, F: one token to several row tiles; whole tiles, ragged ones, odd channels and features
    (1, 1, 1), (1, 384, 1536), (2, 64, 256), (3, 40, 72), (5, 7, 9), (8, 128, 512), (9, 128, 512), (17, 33, 130),
    (127, 128, 128), (128, 64, 64), (129, 136, 264), (300, 256, 512), (257, 100, 397), (1000, 16, 24), (640, 384, 640),
]


@pytest.mark.parametrize("dt", [BF16, FP16, FP32], ids=lambda d: str(d)[6:])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_matches_oracle(shape, dt):
    M, C, F = shape
    act = "gelu" if (M + C + F) % 2 else "silu"
    check(*make(M, C, F, dt, seed=M + C + F), act, f"{shape} {dt} {act}")


@pytest.mark.parametrize("dt", [BF16, FP16, FP32], ids=lambda d: str(d)[6:])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_both_activations(act, dt):
    check(*make(200, 96, 160, dt, seed=5), act, f"{act} {dt}")


@pytest.mark.parametrize("waves,C,F", [(5, 16, 1200), (3, 136, 1200)])
def test_more_rows_than_one_chunk(waves, C, F):
    """Rows are taken in chunks (of whole waves of 148 128-row tiles); the weight
    gradients add up over them."""
    M = waves * 18944 + 300
    assert evo.evo_transition_bwd_workspace_size(M, C, F, evo.EVO_DTYPE_BF16) == \
        evo.evo_transition_bwd_workspace_size(M + 18944, C, F, evo.EVO_DTYPE_BF16)
    check(*make(M, C, F, BF16, seed=1), "silu", f"chunks {M}")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("shape", [(100, 128, 512), (509, 96, 130), (3000, 35, 130), (1300, 101, 397), (2000, 128, 512)], ids=str)
def test_fp32_rows_in_groups_and_in_tiles(shape, act):
    check(*make(*shape, FP32, seed=shape[0]), act, f"{shape} {act}")


@pytest.mark.parametrize("M,C,F,dt", [(19244, 16, 1200, FP32), (57100, 132, 1201, FP16), (94820, 17, 1201, BF16),
                                      (2100000, 9, 8, FP16)], ids=str)
def test_chunks_of_every_form(M, C, F, dt):
    """Several chunks with fp32, and with copies of rows that are no whole 16-byte units."""
    check(*make(M, C, F, dt, seed=M), "silu", f"chunks {M} {C} {F} {dt}")


def test_more_row_tiles_than_a_grid_dimension():
    """More than 65535 tiles of 128 rows, with one feature in fp32 (one chunk by bytes alone)."""
    M = 65536 * 128 + 1000
    x, wg, wu, wd, dy = make(M, 2, 1, FP32, seed=3)
    y = evo.transition(x, wg, wu, wd)
    dx, *dw = evo.transition_backward(x, wg, wu, wd, dy)
    assert evo.evo_attn_sync_status() == evo.EVO_OK
    at = torch.cat([torch.arange(0, M, 50021), torch.arange(M - 1200, M)])
    ref, err = T.forward(x[at], wg, wu, wd, "silu", FP32)
    within(y[at], ref, err, "y")
    ref, err = T.backward(x, wg, wu, wd, dy, "silu", FP32)
    for name, g, r, e in zip(("dx", "dw_gate", "dw_up", "dw_down"), (dx, *dw), ref, err):
        within(g, r, e, name)


@pytest.mark.parametrize("shape,dt", [((8321, 128, 512), BF16), ((8200, 40, 72), FP16), ((19100, 256, 304), BF16),
                                      ((20001, 192, 136), FP16), ((8193, 100, 130), BF16), ((38000, 64, 128), BF16),
                                      ((9000, 250, 400), FP16), ((8193, 1, 1), BF16), ((60000, 64, 64), BF16),
                                      ((60001, 128, 40), FP16), ((60000, 96, 192), BF16), ((40000, 136, 100), BF16)], ids=str)
def test_many_rows_of_few_channels(shape, dt):
    """Sizes at which Y of a row tile is formed without the [M, F] array: one and
    several tiles a CTA, one and several feature chunks, C up to 128 and up to 256."""
    M, C, F = shape
    act = "gelu" if M % 2 else "silu"
    x, wg, wu, wd, _ = make(M, C, F, dt, seed=M)
    y = evo.transition(x, wg, wu, wd, act=act)
    assert evo.evo_attn_sync_status() == evo.EVO_OK
    ref, err = T.forward(x, wg, wu, wd, act, dt)
    within(y, ref, err, f"{shape} {dt}")
    assert torch.equal(evo.transition(x, wg, wu, wd, act=act), y)


@pytest.mark.parametrize("C,F", [(256, 1024), (192, 512), (128, 512), (64, 256)])
def test_msa_size(C, F):
    """Long runs of chunks in every CTA (131072 rows, the MSA of 512 sequences of 256
    residues): sampled rows against the oracle, repeated calls to the bit."""
    x, wg, wu, wd, _ = make(512 * 256, C, F, BF16, seed=C)
    y = evo.transition(x, wg, wu, wd)
    assert evo.evo_attn_sync_status() == evo.EVO_OK
    at = torch.arange(0, 512 * 256, 251)
    ref, err = T.forward(x[at], wg, wu, wd, "silu", BF16)
    within(y[at], ref, err, f"{C} {F}")
    for _ in range(5):
        assert torch.equal(evo.transition(x, wg, wu, wd), y)
    assert evo.evo_attn_sync_status() == evo.EVO_OK


@pytest.mark.parametrize("shape,dt", [((8321, 128, 512), BF16), ((8200, 40, 72), FP16), ((20001, 64, 264), BF16),
                                      ((8193, 100, 130), BF16), ((38000, 128, 128), FP16), ((8193, 1, 1), BF16),
                                      ((60000, 128, 300), BF16), ((20000, 200, 264), BF16)], ids=str)
def test_backward_many_rows_of_few_channels(shape, dt):
    """Long row counts over narrow blocks: ragged tiles in every direction, all
    gradients and each side alone."""
    M, C, F = shape
    act = "gelu" if M % 2 else "silu"
    x, wg, wu, wd, dy = make(M, C, F, dt, seed=M)
    grads = evo.transition_backward(x, wg, wu, wd, dy, act=act)
    assert evo.evo_attn_sync_status() == evo.EVO_OK
    ref, err = T.backward(x, wg, wu, wd, dy, act, dt)
    for name, g, r, e in zip(("dx", "dw_gate", "dw_up", "dw_down"), grads, ref, err):
        within(g, r, e, f"{shape} {dt} {name}")
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(evo.transition_backward(x, wg, wu, wd, dy, act=act), grads))
    assert torch.equal(evo.transition_backward(x, wg, wu, wd, dy, act=act, need_dw=False)[0], grads[0])
    none, *dw = evo.transition_backward(x, wg, wu, wd, dy, act=act, need_dx=False)
    assert none is None and all(torch.equal(a, b) for a, b in zip(dw, grads[1:]))
    assert evo.evo_attn_sync_status() == evo.EVO_OK


def test_activation_range():
    """Gates far out on both sides: no overflow on the way to 0 or to g."""
    gates = torch.tensor([-1e30, -3e4, -100.0, -88.5, -87.0, -20.0, -1.0, -0.0, 1e-30, 20.0, 100.0, 1e3])
    for dt in (BF16, FP32):
        x = torch.zeros(12, 16)
        x[:, 0], x[:, 1] = gates, 1.0
        wg, wu, wd = torch.zeros(16, 16), torch.zeros(16, 16), torch.eye(16)
        wg[:, 0], wu[:, 1] = 1.0, 1.0
        x, wg, wu, wd = (t.to(dt).cuda() for t in (x, wg, wu, wd))
        for act in ("silu", "gelu"):
            y = evo.transition(x, wg, wu, wd, act=act)
            ref, err = T.forward(x, wg, wu, wd, act, dt)
            # far tails come out below the type's normal numbers
            assert np.all(np.abs(T._f64(y) - ref) <= err + 2.0 ** -100), (dt, act)


@pytest.mark.parametrize("M", [1, 40])
def test_nan_stays_in_its_row(M):
    x, wg, wu, wd, _ = make(M + 1, 64, 128, BF16, seed=2)
    clean = evo.transition(x, wg, wu, wd)
    x[M, 3] = float("nan")
    y = evo.transition(x, wg, wu, wd)
    assert torch.isnan(y[M]).all() and torch.equal(y[:M], clean[:M])


def test_empty_sizes():
    x, wg, wu, wd, dy = make(4, 16, 24, BF16, seed=0)
    assert evo.transition(x[:0], wg, wu, wd).shape == (0, 16)
    dx, *dw = evo.transition_backward(x[:0], wg, wu, wd, dy[:0])
    assert dx.shape == (0, 16) and all((g == 0).all() for g in dw)
    none = torch.empty(0, 16, dtype=BF16, device="cuda")
    y = evo.transition(x, none, none, none.T.contiguous(), out=torch.full_like(x, 7))
    assert (y == 0).all()
    dx, *_ = evo.transition_backward(x, none, none, none.T.contiguous(), dy)
    assert (dx == 0).all()


def test_only_the_asked_gradients():
    x, wg, wu, wd, dy = make(300, 64, 96, BF16, seed=4)
    full = evo.transition_backward(x, wg, wu, wd, dy)
    dx, *none = evo.transition_backward(x, wg, wu, wd, dy, need_dw=False)
    assert none == [None] * 3 and torch.equal(dx, full[0])
    none, *dw = evo.transition_backward(x, wg, wu, wd, dy, need_dx=False)
    assert none is None and all(torch.equal(a, b) for a, b in zip(dw, full[1:]))
    # one weight's gradient alone, through the C entry point
    M, C, F = 300, 64, 96
    ws = torch.empty(evo.evo_transition_bwd_workspace_size(M, C, F, 0), dtype=torch.uint8, device="cuda")
    for i in range(3):
        out = [None] * 3
        out[i] = torch.full_like((wg, wu, wd)[i], 9)
        st = evo.evo_transition_bwd(x.data_ptr(), wg.data_ptr(), wu.data_ptr(), wd.data_ptr(), dy.data_ptr(), None,
                                    *(None if o is None else o.data_ptr() for o in out), ws.data_ptr(), ws.numel(), M, C,
                                    F, 0, evo.EVO_DTYPE_BF16, None)
        torch.cuda.synchronize()
        assert st == evo.EVO_OK and torch.equal(out[i], full[1 + i])


@pytest.mark.parametrize("dt", [BF16, FP32], ids=lambda d: str(d)[6:])
@pytest.mark.parametrize("shape", [(4, 64, 128), (700, 72, 200)], ids=str)
def test_same_bits_every_time_and_writes_only_its_rows(shape, dt):
    M, C, F = shape
    x, wg, wu, wd, dy = make(M, C, F, dt, seed=6)
    out = torch.full((M + 3, C), 5.0, dtype=dt, device="cuda")
    y = evo.transition(x, wg, wu, wd, out=out[:M])
    assert (out[M:] == 5).all()
    g = evo.transition_backward(x, wg, wu, wd, dy)
    for _ in range(3):
        assert torch.equal(evo.transition(x, wg, wu, wd), y)
        assert all(torch.equal(a, b) for a, b in zip(evo.transition_backward(x, wg, wu, wd, dy), g))


def test_leading_axes_are_rows():
    x, wg, wu, wd, dy = make(24, 32, 64, FP16, seed=7)
    y = evo.transition(x, wg, wu, wd)
    assert torch.equal(evo.transition(x.view(2, 3, 4, 32), wg, wu, wd), y.view(2, 3, 4, 32))
    assert torch.equal(evo.transition(x[0], wg, wu, wd), evo.transition(x[:1], wg, wu, wd)[0])
    dx, *_ = evo.transition_backward(x.view(2, 12, 32), wg, wu, wd, dy.view(2, 12, 32))
    assert dx.shape == (2, 12, 32)


def test_unaligned_tensors():
    """2-byte aligned tensors run where C or F is no multiple of 8, and are refused elsewhere."""
    def shifted(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
        buf[1:] = t.flatten()
        return buf[1:].view(t.shape)
    check(*(shifted(t) for t in make(140, 50, 70, BF16, seed=8)), "silu", "unaligned")
    check(*(shifted(t) for t in make(140, 48, 64, FP32, seed=8)), "silu", "unaligned fp32")
    check(*(shifted(t) for t in make(3, 50, 70, BF16, seed=8)), "silu", "unaligned, few rows")
    x, wg, wu, wd, _ = make(140, 48, 64, BF16, seed=8)
    with pytest.raises(evo.EvoAttnError) as e:
        evo.transition(shifted(x), wg, wu, wd)
    assert e.value.status == evo.EVO_ERR_MISALIGNED


def test_another_stream_and_two_calls_at_once():
    side = torch.cuda.Stream()
    a, b = make(600, 128, 256, BF16, seed=9), make(600, 128, 256, BF16, seed=10)
    torch.cuda.synchronize()
    check(*a, "silu", "side stream", stream=side)
    wants = [evo.transition(*t[:4]) for t in (a, b)]
    torch.cuda.synchronize()
    for _ in range(10):
        y0 = evo.transition(*a[:4], stream=side)
        y1 = evo.transition(*b[:4])
        torch.cuda.synchronize()
        assert torch.equal(y0, wants[0]) and torch.equal(y1, wants[1])


@pytest.mark.parametrize("shape,dt", [((1, 384, 512), BF16), ((500, 64, 96), BF16), ((500, 50, 70), FP16),
                                      ((130, 32, 48), FP32)], ids=str)
def test_replays_in_a_cuda_graph(shape, dt):
    M, C, F = shape
    first, second = make(M, C, F, dt, seed=11), make(M, C, F, dt, seed=12)
    bufs = [t.clone() for t in first]
    evo.transition(*bufs[:4])
    evo.transition_backward(*bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = evo.transition(*bufs[:4])
        grads = evo.transition_backward(*bufs)
    for case in (second, first):
        for buf, t in zip(bufs, case):
            buf.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert evo.evo_attn_sync_status() == evo.EVO_OK
        assert torch.equal(y, evo.transition(*case[:4]))
        assert all(torch.equal(a, b) for a, b in zip(grads, evo.transition_backward(*case)))
