"""Transition and relative-position entry points: bad arguments come back with
the documented status codes (or Python errors) before anything touches a GPU."""
import pytest
import torch

import triangle_biased_attention_b200 as evo
from triangle_biased_attention_b200 import build as evo_build

FAR = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def lib():
    evo_build.build()
    return evo.load_library()


def fwd(M=16, C=304, F=64, act=0, dt=evo.EVO_DTYPE_BF16, Wb=None, **kw):
    a = dict(X=1 * FAR, Wg=2 * FAR, Wu=3 * FAR, Wd=4 * FAR, Y=5 * FAR, W=6 * FAR)
    a.update(kw)
    if Wb is None:
        Wb = max(0, evo.evo_transition_fwd_workspace_size(M, C, F, dt))
    return evo.evo_transition_fwd(a["X"], a["Wg"], a["Wu"], a["Wd"], a["Y"], a["W"], Wb, M, C, F, act, dt, None)


def bwd(M=16, C=304, F=64, act=0, dt=evo.EVO_DTYPE_BF16, Wb=None, **kw):
    a = dict(X=1 * FAR, Wg=2 * FAR, Wu=3 * FAR, Wd=4 * FAR, dY=5 * FAR, dX=6 * FAR, dWg=7 * FAR, dWu=8 * FAR,
             dWd=9 * FAR, W=10 * FAR)
    a.update(kw)
    if Wb is None:
        Wb = max(0, evo.evo_transition_bwd_workspace_size(M, C, F, dt))
    return evo.evo_transition_bwd(a["X"], a["Wg"], a["Wu"], a["Wd"], a["dY"], a["dX"], a["dWg"], a["dWu"], a["dWd"],
                                  a["W"], Wb, M, C, F, act, dt, None)


# without a GPU these made-up addresses are refused as not device memory, after every other check
ACCEPTED = evo.EVO_ERR_INVALID_ARG


def test_transition_workspace_size():
    for size in (evo.evo_transition_fwd_workspace_size, evo.evo_transition_bwd_workspace_size):
        assert size(16, 304, 64, evo.EVO_DTYPE_BF16) > 0
        assert size(-1, 32, 64, 0) == evo.EVO_ERR_INVALID_ARG
        assert size(16, 32, 64, 9) == evo.EVO_ERR_UNSUPPORTED_DTYPE
        assert size(1 << 31, 32, 64, 0) == evo.EVO_ERR_UNSUPPORTED_SHAPE
        assert size(16, (1 << 20) + 1, 64, 0) == evo.EVO_ERR_UNSUPPORTED_SHAPE
        assert size(0, 32, 64, 0) == 0 and size(16, 0, 64, 0) == 0 and size(16, 32, 0, 0) == 0
        # the workspace holds chunks of rows, not all of them
        for C in (128, 304):
            assert size(1 << 24, C, 512, 0) == size(1 << 30, C, 512, 0) < 1 << 30
    # the one-kernel forward needs none, and takes a NULL for it
    assert evo.evo_transition_fwd_workspace_size(1 << 20, 128, 512, evo.EVO_DTYPE_FP16) == 0
    assert fwd(M=1 << 20, C=128, F=512, W=None, Y=5 * FAR + 2) == evo.EVO_ERR_MISALIGNED


@pytest.mark.parametrize("call", [fwd, bwd])
def test_transition_checks_arguments(call):
    assert call(C=0) == evo.EVO_OK
    assert call(F=0) == ACCEPTED and call(C=1, F=1) == ACCEPTED
    assert call(M=-1, Wb=0) == evo.EVO_ERR_INVALID_ARG
    assert call(act=2) == evo.EVO_ERR_INVALID_ARG
    assert call(dt=3, Wb=1 << 20) == evo.EVO_ERR_UNSUPPORTED_DTYPE
    assert call(Wb=-1) == evo.EVO_ERR_INVALID_ARG
    for name in ("X", "Wg", "Wu", "Wd", "W"):
        assert call(**{name: None}) == evo.EVO_ERR_INVALID_ARG
    assert call(C=1 << 21, Wb=0) == evo.EVO_ERR_UNSUPPORTED_SHAPE
    assert call(M=1 << 31, Wb=0) == evo.EVO_ERR_UNSUPPORTED_SHAPE
    assert call() == ACCEPTED
    # alignment: 16 bytes when C and F are multiples of 8, else the element's
    assert call(X=FAR + 8) == evo.EVO_ERR_MISALIGNED
    assert call(Wd=4 * FAR + 2) == evo.EVO_ERR_MISALIGNED
    assert call(C=33, X=FAR + 2) == ACCEPTED and call(F=60, X=FAR + 2) == ACCEPTED
    assert call(C=33, X=FAR + 1) == evo.EVO_ERR_MISALIGNED
    assert call(dt=evo.EVO_DTYPE_FP32, X=FAR + 4) == ACCEPTED
    assert call(dt=evo.EVO_DTYPE_FP32, X=FAR + 2) == evo.EVO_ERR_MISALIGNED
    assert call(W=6 * FAR + 16 if call is fwd else 10 * FAR + 16) == evo.EVO_ERR_MISALIGNED


def test_transition_overlaps_and_workspace():
    full = evo.evo_transition_fwd_workspace_size(16, 304, 64, 0)
    # a short workspace or an overlap is refused like a made-up pointer, so each is checked
    # with an alignment fault behind it that an accepted call would report instead
    assert fwd(Y=5 * FAR + 2, W=6 * FAR) == evo.EVO_ERR_MISALIGNED
    assert fwd(Wb=full - 1, Y=5 * FAR + 2) == evo.EVO_ERR_INVALID_ARG
    assert fwd(Y=FAR) == evo.EVO_ERR_INVALID_ARG
    assert bwd(dX=FAR) == evo.EVO_ERR_INVALID_ARG
    assert bwd(dX=None, dWg=None, dWu=None, dWd=None) == evo.EVO_OK
    assert bwd(M=0, dWg=None, dWu=None, dWd=None) == evo.EVO_OK


def rel(B=2, Sq=5, Sk=7, H=3, nb=9, dt=evo.EVO_DTYPE_BF16, **kw):
    a = dict(table=FAR, borders=2 * FAR, pq=3 * FAR, pk=4 * FAR, cq=None, ck=None, base=None, pair=5 * FAR)
    a.update(kw)
    return evo.evo_relpos_fwd(a["table"], a["borders"], a["pq"], a["pk"], a["cq"], a["ck"], a["base"], a["pair"], B, Sq,
                              Sk, H, nb, dt, None)


def rel_bwd(B=2, Sq=5, Sk=7, H=3, nb=9, dt=evo.EVO_DTYPE_BF16, Wb=1 << 30, **kw):
    a = dict(dpair=FAR, borders=2 * FAR, pq=3 * FAR, pk=4 * FAR, cq=None, ck=None, dtable=5 * FAR, W=6 * FAR)
    a.update(kw)
    return evo.evo_relpos_bwd(a["dpair"], a["borders"], a["pq"], a["pk"], a["cq"], a["ck"], a["dtable"], a["W"], Wb, B,
                              Sq, Sk, H, nb, dt, None)


@pytest.mark.parametrize("call", [rel, rel_bwd])
def test_relpos_checks_arguments(call):
    assert call() == ACCEPTED
    assert call(H=0) == evo.EVO_OK
    assert call(B=-1) == evo.EVO_ERR_INVALID_ARG
    assert call(nb=-1) == evo.EVO_ERR_INVALID_ARG
    assert call(dt=5) == evo.EVO_ERR_UNSUPPORTED_DTYPE
    assert call(nb=2049) == evo.EVO_ERR_UNSUPPORTED_SHAPE
    assert call(B=1 << 17) == evo.EVO_ERR_UNSUPPORTED_SHAPE
    assert call(Sq=1 << 30) == evo.EVO_ERR_UNSUPPORTED_SHAPE
    assert call(cq=7 * FAR) == evo.EVO_ERR_INVALID_ARG          # chains of one side only
    assert call(pq=3 * FAR + 2) == evo.EVO_ERR_MISALIGNED
    assert call(pq=None) == evo.EVO_ERR_INVALID_ARG and call(borders=None) == evo.EVO_ERR_INVALID_ARG
    assert call(nb=0, borders=None, pq=3 * FAR + 2) == evo.EVO_ERR_MISALIGNED     # no border to point at


def test_relpos_specific_refusals():
    assert rel(Sq=0) == evo.EVO_OK and rel(B=0, table=None) == evo.EVO_OK
    assert rel(table=FAR + 1) == evo.EVO_ERR_MISALIGNED
    assert rel(pair=FAR) == evo.EVO_ERR_INVALID_ARG
    assert rel_bwd(dtable=None) == evo.EVO_ERR_INVALID_ARG
    assert rel_bwd(Wb=3) == evo.EVO_ERR_INVALID_ARG
    assert rel_bwd(W=6 * FAR + 8) == evo.EVO_ERR_MISALIGNED
    assert evo.evo_relpos_bwd_workspace_size(1, 0, 7, 3, 9, 0) == 0
    assert evo.evo_relpos_bwd_workspace_size(1, -1, 7, 3, 9, 0) == evo.EVO_ERR_INVALID_ARG
    assert evo.evo_relpos_bwd_workspace_size(1, 9, 7, 3, 4000, 0) == evo.EVO_ERR_UNSUPPORTED_SHAPE
    assert evo.evo_relpos_bwd_workspace_size(1, 9, 7, 3, 9, 1) >= 3 * 11 * 4


def test_transition_wrapper_validates_before_calling():
    x, w, wd = torch.zeros(4, 8), torch.zeros(16, 8), torch.zeros(8, 16)
    with pytest.raises(ValueError, match="CUDA"):
        evo.transition(x, w, w, wd)
    with pytest.raises(ValueError, match="CUDA"):
        evo.transition_backward(x, w, w, wd, x)
    with pytest.raises(ValueError, match="w_down"):
        evo.transition(x, w, w, w)
    with pytest.raises(ValueError, match="w_up"):
        evo.transition(x, w, w[:8], wd)
    with pytest.raises(TypeError):
        evo.transition(x.double(), w.double(), w.double(), wd.double())
    with pytest.raises(TypeError):
        evo.transition(x, w.half(), w, wd)
    with pytest.raises(ValueError, match="contiguous"):
        evo.transition(torch.zeros(8, 4).T, w, w, wd)
    with pytest.raises(ValueError, match="act"):
        evo.transition(x, w, w, wd, act="relu")
    with pytest.raises(ValueError, match="dy"):
        evo.transition_backward(x, w, w, wd, x[:2])


def test_relpos_wrapper_validates_before_calling():
    borders = evo.relpos_clip_borders(2)
    pos = torch.zeros(1, 6, dtype=torch.int32)
    table = torch.zeros(6, 4)
    with pytest.raises(ValueError, match="CUDA"):
        evo.relpos_bias(table, borders, pos)
    with pytest.raises(ValueError, match="table"):
        evo.relpos_bias(table, borders, pos, chain=pos)       # chains need one more row
    with pytest.raises(TypeError, match="pos"):
        evo.relpos_bias(table, borders, pos.long())
    with pytest.raises(TypeError, match="borders"):
        evo.relpos_bias(table, borders.float(), pos)
    with pytest.raises(ValueError, match="together"):
        evo.relpos_bias(table, borders, pos, pos, chain=pos)
    with pytest.raises(ValueError, match="without pos_k"):
        evo.relpos_bias(table, borders, pos, chain=pos, chain_k=pos.clone())
    with pytest.raises(ValueError, match="base"):
        evo.relpos_bias(table, borders, pos, base=torch.zeros(1, 4, 6, 6))
    with pytest.raises(ValueError, match="dpair"):
        evo.relpos_bias_backward(torch.zeros(1, 4, 6, 6), borders, pos)
    with pytest.raises(ValueError, match="CUDA"):
        evo.relpos_bias_backward(torch.zeros(1, 1, 4, 6, 6), borders, pos)
