"""lce_f64 of lce_oracle.py for full-size heads (TEST INFRASTRUCTURE): the same
definition in the same row blocks, its row-wise steps on all host cores. numpy
runs them on one, which is most of the time of a case of 10^9 logits. Every
number and every sum is formed in the same order: the results are lce_f64's,
bit for bit.
"""
from __future__ import annotations

import math

import numpy as np

from ._rows import by_rows
from .lce_oracle import IGNORE_INDEX, MEAN, _prepare

LARGE = 1 << 27   # logits from which on lce_bf16 comes here


def lce_large_f64(H, W, y, *, ignore_index=IGNORE_INDEX, reduction=MEAN, n_valid_override=-1, grad_loss=1.0, row_block=256,
                  grads=True):
    """lce_f64."""
    H = np.asarray(H, dtype=np.float64)
    W = np.asarray(W, dtype=np.float64)
    N, d = H.shape
    V = W.shape[0]
    y, valid, n, scale, lscale = _prepare(y, V, ignore_index, reduction, n_valid_override, grad_loss)
    lse, loss_i, zt = np.empty(N), np.zeros(N), np.zeros(N)
    dH = np.zeros((N, d)) if grads else None
    dW = np.zeros((V, d)) if grads else None
    for r0 in range(0, N, row_block):
        r1 = min(N, r0 + row_block)
        z = H[r0:r1] @ W.T

        def rows(a, b):   # rows [a, b) of the block; their logits become their gradient
            zr, at = z[a:b], slice(r0 + a, r0 + b)
            m = zr.max(axis=1)
            lse[at] = m + np.log(np.exp(zr - m[:, None]).sum(axis=1))
            v = valid[at]
            yy = np.where(v, y[at], 0)
            zt[at] = np.where(v, zr[np.arange(b - a), yy], 0.0)
            loss_i[at] = np.where(v, lse[at] - zt[at], 0.0)
            if grads:
                p = np.exp(zr - lse[at, None])
                p[np.flatnonzero(v), yy[v]] -= 1.0
                z[a:b] = p * (v * scale)[:, None]

        by_rows(rows, r1 - r0, V)
        if not grads:
            continue
        dH[r0:r1] = z @ W
        more = z.T @ H[r0:r1]
        by_rows(lambda a, b: np.add(dW[a:b], more[a:b], out=dW[a:b]), V, d)
    out = {"loss": math.fsum(loss_i.tolist()) * lscale, "lse": lse, "loss_i": loss_i, "zt": zt, "n_valid": n}
    if grads:
        out["dH"], out["dW"] = dH, dW
    return out
