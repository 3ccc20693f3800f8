"""fp64 CPU oracle for the head's token operators (TEST INFRASTRUCTURE).

Log-probabilities of given tokens with entropy and top alternatives, their
gradient, and the distillation loss with its gradient, written from the
definitions with numpy on whole [N, V] arrays (small cases only).

The gradients come with ``bulk``: the sum of the absolute values of the terms
whose sum the gradient is, dH_bulk = |G| |W| and dW_bulk = |G|^T |H| with |G|
the absolute values of each part of G. A bound on the relative error of every
term, times the bulk, bounds the error of the element. Log-probabilities add
``slack``, the same sums over p |e|: what an absolute error of log p + entropy,
which cancels in confident rows, is multiplied by.
"""
from __future__ import annotations

import numpy as np

from .lce_oracle import IGNORE_INDEX, MEAN


def _head(H, W, temperature):
    z = H @ W.T
    zt = z / temperature
    m = zt.max(axis=1, keepdims=True)
    lse = m + np.log(np.exp(zt - m).sum(axis=1, keepdims=True))
    return z, zt - lse, lse[:, 0]


def _xlogx(p, logp):
    return np.where(p > 0, p * np.where(p > 0, logp, 0.0), 0.0)


def logprobs_f64(H, W, y, *, temperature=1.0, top_k=0, ignore_index=IGNORE_INDEX):
    """logp, lse, entropy [N]; top_logp, top_idx [N, top_k] (ties: the lower index first)."""
    z, logq, lse = _head(H, W, temperature)
    N, V = z.shape
    told = (y != ignore_index) & (y >= 0) & (y < V)
    logp = np.where(told, logq[np.arange(N), np.where(told, y, 0)], 0.0)
    entropy = -_xlogx(np.exp(logq), logq).sum(axis=1)
    order = np.lexsort((np.broadcast_to(np.arange(V), z.shape), -z), axis=1)[:, :top_k]
    return {"logp": logp, "lse": lse, "entropy": entropy, "top_idx": order,
            "top_logp": np.take_along_axis(logq, order, axis=1)}


def logprobs_backward_f64(H, W, y, g_logp, g_entropy, *, temperature=1.0, ignore_index=IGNORE_INDEX):
    """dH, dW of sum_i g_logp_i logp_i + g_entropy_i entropy_i, and their bulks."""
    z, logq, _ = _head(H, W, temperature)
    N, V = z.shape
    p = np.exp(logq)
    ent = -_xlogx(p, logq).sum(axis=1)
    told = (y != ignore_index) & (y >= 0) & (y < V)
    a = np.where(told, g_logp, 0.0)[:, None]
    e = (np.zeros(N) if g_entropy is None else g_entropy)[:, None]
    dev = logq + ent[:, None]
    hot = np.zeros_like(p)
    hot[np.arange(N)[told], y[told]] = 1.0
    G = (hot * a - p * (a + e * dev)) / temperature
    size = (hot * np.abs(a) + p * (np.abs(a) + np.abs(e) * np.abs(dev))) / temperature
    slack = p * np.abs(e) / temperature
    return {"dH": G @ W, "dW": G.T @ H, "dH_bulk": size @ np.abs(W), "dW_bulk": size.T @ np.abs(H),
            "dH_slack": slack @ np.abs(W), "dW_slack": slack.T @ np.abs(H)}


def teacher_f64(idx, t, V, *, temperature=1.0, renormalize=True, ignore_index=IGNORE_INDEX):
    """The teacher's probabilities as a dense [N, V] array, and which rows keep an entry."""
    N, K = idx.shape
    kept = (idx != ignore_index) & (idx >= 0) & (idx < V) & (t > -np.inf)
    q = np.zeros((N, K))
    for i in range(N):
        if not kept[i].any():
            continue
        if renormalize:
            s = t[i, kept[i]] / temperature
            w = np.exp(s - s.max())
            q[i, kept[i]] = w / w.sum()
        else:
            q[i, kept[i]] = np.exp(t[i, kept[i]])
    dense = np.zeros((N, V))
    for i in range(N):
        np.add.at(dense[i], idx[i, kept[i]], q[i, kept[i]])
    return q, dense, kept


def distill_f64(H, W, idx, t, *, temperature=1.0, renormalize=True, ignore_index=IGNORE_INDEX, reduction=MEAN,
                n_valid_override=-1, grad_loss=1.0):
    """loss, row_loss [N], dH, dW and the gradients' bulks. An index that occurs
    twice in a row adds q log q of each entry to the loss."""
    z, logq, _ = _head(H, W, temperature)
    q, dense, kept = teacher_f64(idx, t, z.shape[1], temperature=temperature, renormalize=renormalize,
                                 ignore_index=ignore_index)
    safe = np.where(kept, idx, 0)
    at = np.take_along_axis(logq, safe, axis=1)
    terms = np.where(q > 0, q * (np.log(np.where(q > 0, q, 1.0)) - at), 0.0)
    row = temperature ** 2 * terms.sum(axis=1)
    n = n_valid_override if n_valid_override >= 0 else int(kept.any(axis=1).sum())
    w = (1.0 / n if n > 0 else 0.0) if reduction == MEAN else 1.0
    m = q.sum(axis=1, keepdims=True)
    f = grad_loss * w * temperature
    p = np.exp(logq)
    G = f * (m * p - dense)
    size = abs(f) * (m * p + dense)
    return {"loss": row.sum() * w, "row_loss": row, "dH": G @ W, "dW": G.T @ H,
            "dH_bulk": size @ np.abs(W), "dW_bulk": size.T @ np.abs(H)}
