"""The relative-position bias and its table gradient on the GPU against the
float64 oracle.

Forward: without a base the exact table values; with one, an fp32 sum (exact
table and base, one rounding of 2^-24) rounded to the type.  Backward: sums of
exact fp32 values in a chain of at most DEPTH additions (a thread's rows, its
flushes, the tile's columns and the tiles), then one rounding to the type.
"""
import numpy as np
import pytest
import torch

import triangle_biased_attention_b200 as evo
from oracle import relpos as R
from oracle.transition import _f64, units

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
DEPTH = 4096
DEV = "cuda:0"


def make(B, Sq, Sk, H, nb, dt, seed, chains=False, spread=None, same=False):
    g = torch.Generator().manual_seed(seed)
    spread = spread or 3 * nb + 4
    borders = torch.randperm(2 * spread, generator=g)[:nb].sort().values.to(torch.int32) - spread
    ints = lambda n, hi: torch.randint(-hi, hi + 1, (B, n), generator=g).to(torch.int32)  # noqa: E731
    pq, pk = ints(Sq, spread), ints(Sk, spread)
    cq, ck = (ints(Sq, 1), ints(Sk, 1)) if chains else (None, None)
    if same:
        pq = torch.arange(Sq, dtype=torch.int32).repeat(B, 1)
        pk = torch.arange(Sk, dtype=torch.int32).repeat(B, 1)
    table = torch.randn(nb + 1 + chains, H, generator=g).to(dt)
    pair = torch.randn(B, 1, H, Sq, Sk, generator=g).to(dt)
    on = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    return [on(t) for t in (table, borders, pq, pk, cq, ck, pair)]


def check(table, borders, pq, pk, cq, ck, pair, what):
    dt = table.dtype
    r, tiny = units(dt)
    p = evo.relpos_bias(table, borders, pq, pk, cq, ck)
    with_base = evo.relpos_bias(table, borders, pq, pk, cq, ck, base=pair)
    dtable = evo.relpos_bias_backward(pair, borders, pq, pk, cq, ck)
    assert evo.evo_attn_sync_status() == evo.EVO_OK
    assert np.array_equal(_f64(p), R.forward(table, borders, pq, pk, cq, ck)), what
    ref = R.forward(table, borders, pq, pk, cq, ck, pair)
    assert np.all(np.abs(_f64(with_base) - ref) <= (r + 2.0 ** -24) * (1 + 2.0 ** -7) * np.abs(ref) + tiny), what
    args = (table.shape[0], borders, pq, pk, cq, ck)
    ref, size = R.backward(pair, *args), R.backward(pair.abs(), *args)
    gamma = DEPTH * 2.0 ** -24 / (1 - DEPTH * 2.0 ** -24)
    err = gamma * size + r * (np.abs(ref) + gamma * size) + tiny
    got = _f64(dtable)
    print(f"{what}: dtable max err/bound {float((np.abs(got - ref) / np.maximum(err, 1e-300)).max(initial=0)):.3f}")
    assert np.all(np.abs(got - ref) <= err), what
    assert np.all(got[size == 0] == 0), what


SHAPES = [
    # B, Sq, Sk, H, borders
    (1, 1, 1, 1, 0), (1, 1, 1, 3, 1), (2, 5, 7, 3, 5), (1, 1, 1000, 4, 30), (1, 300, 1, 2, 9), (1, 64, 64, 8, 65),
    (2, 130, 264, 5, 65), (1, 257, 513, 16, 31), (3, 100, 1032, 4, 65), (1, 33, 2049, 2, 255), (1, 40, 72, 9, 256),
    (1, 200, 208, 2, 600), (1, 50, 56, 1, 2048), (1, 700, 704, 4, 65),
]


@pytest.mark.parametrize("dt", [BF16, FP16, FP32], ids=lambda d: str(d)[6:])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_matches_oracle(shape, dt):
    chains = sum(shape) % 2 == 0
    check(*make(*shape, dt, seed=sum(shape), chains=chains), f"{shape} {dt} chains={chains}")


@pytest.mark.parametrize("dt", [BF16, FP32], ids=lambda d: str(d)[6:])
def test_running_positions(dt):
    """Residue numbers 0 .. S-1: whole stretches of a row in one bucket."""
    for S in (384, 500):
        check(*make(1, S, S, 4, 65, dt, seed=S, chains=True, same=True), f"running {S}")


def test_borders_far_apart():
    """A span of distances too wide for a table of them, and the ends of the 32-bit range."""
    far = 2 ** 31 - 1
    borders = torch.tensor([-far, -5 * 10 ** 8, -3, 0, 7, 10 ** 9, far], dtype=torch.int32, device=DEV)
    pos = torch.tensor([[-far - 1, -far, -10 ** 9, -4, -3, 0, 1, 7, 8, 10 ** 9, far]], dtype=torch.int32, device=DEV)
    table = torch.arange(8.0, device=DEV)[:, None].repeat(1, 2).to(BF16)
    pair = torch.ones(1, 1, 2, 11, 11, dtype=BF16, device=DEV)
    check(table, borders, pos, pos, None, None, pair, "far")
    log = evo.relpos_log_borders(32, 10 ** 6).to(DEV)
    table, _, pq, pk, _, _, pair = make(1, 90, 120, 2, log.numel(), FP32, seed=3, spread=2 * 10 ** 6)
    check(table, log, pq, pk, None, None, pair, "log")


def test_borders_out_of_order_stay_in_bounds():
    table, borders, pq, pk, cq, ck, pair = make(1, 50, 60, 2, 40, FP32, seed=5, chains=True)
    for b in (borders.flip(0).contiguous(), torch.randint(-2 ** 31, 2 ** 31 - 1, (40,), dtype=torch.int32, device=DEV)):
        p = evo.relpos_bias(table, b, pq, pk, cq, ck)
        same = (cq[:, :, None] == ck[:, None, :])[:, None, None].expand_as(p)
        last = table[-1][None, None, :, None, None].expand_as(p)
        assert torch.equal(p[~same], last[~same]) and torch.isin(p, table).all()
        evo.relpos_bias_backward(pair, b, pq, pk, cq, ck)
    assert evo.evo_attn_sync_status() == evo.EVO_OK


def test_infinities_and_nan_keep_their_places():
    table, borders, pq, pk, _, _, pair = make(1, 40, 48, 8, 9, BF16, seed=6)
    table[3, 1], table[2, 0] = float("-inf"), torch.finfo(BF16).min
    pair[0, 0, 2, 5, 6] = float("nan")
    rows = torch.from_numpy(R.rows(borders, pq, pk)).to(DEV)
    assert torch.equal(evo.relpos_bias(table, borders, pq, pk), table[rows].permute(0, 3, 1, 2)[:, None])
    p = evo.relpos_bias(table, borders, pq, pk, base=pair)
    want = (table[rows].permute(0, 3, 1, 2)[:, None].float() + pair.float()).to(BF16)
    assert torch.equal(p.isnan(), want.isnan()) and torch.equal(p.nan_to_num(0), want.nan_to_num(0))
    d = evo.relpos_bias_backward(pair, borders, pq, pk)
    bad = torch.zeros_like(table, dtype=torch.bool)
    bad[rows[0, 5, 6], 2] = True
    assert torch.equal(d.isnan(), bad)


def test_unaligned_tensors():
    def shifted(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
        buf[1:] = t.flatten()
        return buf[1:].view(t.shape)
    for dt in (BF16, FP32):
        table, borders, pq, pk, cq, ck, pair = make(2, 70, 256, 4, 33, dt, seed=7, chains=True)
        check(shifted(table), shifted(borders), shifted(pq), shifted(pk), shifted(cq), shifted(ck), shifted(pair),
              f"unaligned {dt}")
        out = shifted(torch.zeros_like(pair))
        assert torch.equal(evo.relpos_bias(table, borders, pq, pk, cq, ck, out=out),
                           evo.relpos_bias(table, borders, pq, pk, cq, ck))


def test_a_strip_of_rows_and_only_its_elements():
    table, borders, pq, _, cq, _, _ = make(1, 256, 256, 4, 65, BF16, seed=8, chains=True)
    whole = evo.relpos_bias(table, borders, pq, chain=cq)
    buf = torch.full((1, 1, 4, 20, 256), 3.0, dtype=BF16, device=DEV).flatten()
    guard = torch.full((buf.numel() + 64,), 3.0, dtype=BF16, device=DEV)
    out = guard[:buf.numel()].view(1, 1, 4, 20, 256)
    evo.relpos_bias(table, borders, pq[:, 100:120].contiguous(), pq, cq[:, 100:120].contiguous(), cq, out=out)
    assert torch.equal(out, whole[:, :, :, 100:120]) and (guard[buf.numel():] == 3).all()


def test_a_tile_past_32_bit_offsets():
    """One block's rows would hold more than 2^31 elements: few values in them, exact sums."""
    Sq, Sk = 2100, 1 << 20
    borders = torch.tensor([-700000, -5, 0, 5, 1000], dtype=torch.int32, device=DEV)
    pq = torch.arange(Sq, dtype=torch.int32, device=DEV).view(1, -1)
    pk = torch.arange(Sk, dtype=torch.int32, device=DEV).view(1, -1)
    dpair = torch.zeros(1, 1, 1, Sq, Sk, dtype=BF16, device=DEV)
    want = np.zeros(6)
    for n, (i, j) in enumerate([(0, 0), (2099, Sk - 1), (2099, 3), (2048, 2047), (2080, 2084), (2070, 800000), (5, 5), (2098, 2099)]):
        dpair[0, 0, 0, i, j] = float(n + 1)
        want[np.searchsorted(borders.cpu().numpy(), i - j, side="right")] += n + 1
    dtable = evo.relpos_bias_backward(dpair, borders, pq, pk)
    assert evo.evo_attn_sync_status() == evo.EVO_OK
    assert np.array_equal(_f64(dtable)[:, 0], want)


def test_empty_sizes():
    table, borders, pq, pk, _, _, pair = make(2, 6, 8, 3, 5, FP32, seed=9)
    assert evo.relpos_bias(table, borders, pq[:, :0].contiguous(), pk).numel() == 0
    d = evo.relpos_bias_backward(pair[:, :, :, :0].contiguous(), borders, pq[:, :0].contiguous(), pk)
    assert d.shape == table.shape and (d == 0).all()


@pytest.mark.parametrize("dt", [BF16, FP32], ids=lambda d: str(d)[6:])
def test_same_bits_streams_and_graph(dt):
    args = make(1, 300, 304, 4, 65, dt, seed=10, chains=True)
    pair, side = args[6], torch.cuda.Stream()
    p, d = evo.relpos_bias(*args[:6]), evo.relpos_bias_backward(pair, *args[1:6])
    torch.cuda.synchronize()
    p2, d2 = evo.relpos_bias(*args[:6], stream=side), evo.relpos_bias_backward(pair, *args[1:6], stream=side)
    side.synchronize()
    assert torch.equal(p, p2) and torch.equal(d, d2)
    bufs = [t.clone() for t in args]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p3, d3 = evo.relpos_bias(*bufs[:6]), evo.relpos_bias_backward(bufs[6], *bufs[1:6])
    other = make(1, 300, 304, 4, 65, dt, seed=11, chains=True)
    for case in (other, args):
        for buf, t in zip(bufs, case):
            buf.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(p3, evo.relpos_bias(*case[:6]))
        assert torch.equal(d3, evo.relpos_bias_backward(case[6], *case[1:6]))
