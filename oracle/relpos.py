"""Float64 oracle for the learned relative-position bias and its table gradient
(test infrastructure only; shares nothing with the CUDA path).

    r(b, i, j)      = the number of borders <= pos_q[b, i] - pos_k[b, j], or the
                      last row where the chains differ
    P[b, 0, h, i, j] = table[r, h] (+ base)
    dtable[r, h]    = sum of dP over the pairs with that row

Pinned in tests/test_relpos_oracle.py by scalar loops and central differences.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle.transition import _f64


def _i64(x):
    return x.detach().cpu().to(torch.int64).numpy() if isinstance(x, torch.Tensor) else np.asarray(x, dtype=np.int64)


def rows(borders, pos_q, pos_k, chain_q=None, chain_k=None) -> np.ndarray:
    """r [B, Sq, Sk]."""
    borders, pos_q, pos_k = _i64(borders), _i64(pos_q), _i64(pos_k)
    d = np.clip(pos_q[:, :, None] - pos_k[:, None, :], -2 ** 31, 2 ** 31 - 1)
    r = np.zeros(d.shape, dtype=np.int64)
    for border in borders:
        r += d >= border
    if chain_q is not None:
        r[_i64(chain_q)[:, :, None] != _i64(chain_k)[:, None, :]] = len(borders) + 1
    return r


def forward(table, borders, pos_q, pos_k, chain_q=None, chain_k=None, base=None) -> np.ndarray:
    r = rows(borders, pos_q, pos_k, chain_q, chain_k)
    p = np.moveaxis(_f64(table)[r], -1, 1)[:, None]
    return p if base is None else p + _f64(base)


def backward(dpair, num_rows, borders, pos_q, pos_k, chain_q=None, chain_k=None) -> np.ndarray:
    r = rows(borders, pos_q, pos_k, chain_q, chain_k)
    dp = _f64(dpair)[:, 0]  # [B, H, Sq, Sk]
    out = np.zeros((num_rows, dp.shape[1]))
    for h in range(dp.shape[1]):
        out[:, h] = np.bincount(r.ravel(), weights=dp[:, h].ravel(), minlength=num_rows)
    return out
