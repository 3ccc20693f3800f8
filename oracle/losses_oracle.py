"""fp64 CPU oracle for the losses on log-probabilities and the layer norm
(TEST INFRASTRUCTURE), written from the definitions with numpy on whole arrays
(small cases only). ``bulk`` as in tokens_oracle.py: the sum of the absolute
values of the terms a gradient is made of.
"""
from __future__ import annotations

import numpy as np

from ._rows import by_rows
from .lce_oracle import IGNORE_INDEX, MEAN
from .tokens_oracle import _head


def _given(y, V, ignore_index):
    return (y != ignore_index) & (y >= 0) & (y < V)


def head_gradients_f64(H, W, y, a, *, temperature=1.0, ignore_index=IGNORE_INDEX):
    """dH, dW and bulks of a loss whose derivative by row i's log-probability is a_i (0 where none is given)."""
    _, logq, _ = _head(H, W, temperature)
    told = _given(y, W.shape[0], ignore_index)
    a = np.where(told, a, 0.0)[:, None]
    G, size = logq, np.empty_like(logq)

    def rows(lo, hi):
        p, given = np.exp(logq[lo:hi]), told[lo:hi]
        hot = np.zeros_like(p)
        hot[np.flatnonzero(given), y[lo:hi][given]] = 1.0
        G[lo:hi] = (hot - p) * a[lo:hi] / temperature
        size[lo:hi] = (hot + p) * np.abs(a[lo:hi]) / temperature

    by_rows(rows, *logq.shape)
    return {"dH": G @ W, "dW": G.T @ H, "dH_bulk": size @ np.abs(W), "dW_bulk": size.T @ np.abs(H)}


def _weight(count, reduction, n_valid_override):
    n = n_valid_override if n_valid_override >= 0 else count
    return (1.0 / n if n > 0 else 0.0) if reduction == MEAN else 1.0


def policy_rows_f64(logp, told, advantages, old_logp=None, ref_logp=None, weights=None, *, clip_low=0.2, clip_high=0.2,
                    dual_clip=0.0, kl="none", kl_coef=0.0):
    """row_loss and its derivative by logp."""
    row, slope = np.zeros(len(logp)), np.zeros(len(logp))
    for i in range(len(logp)):
        w = 1.0 if weights is None else weights[i]
        if not told[i] or w == 0.0:
            continue
        A, gain, s = advantages[i], 0.0, 0.0
        if A != 0.0:
            r = 1.0 if old_logp is None else np.exp(logp[i] - old_logp[i])
            free, bound = r * A, min(max(r, 1.0 - clip_low), 1.0 + clip_high) * A
            gain, s = (bound, 0.0) if bound < free else (free, free)
            if A < 0 and dual_clip > 0 and gain < dual_clip * A:
                gain, s = dual_clip * A, 0.0
        row[i], slope[i] = -gain, -s
        if kl != "none":
            u = logp[i] - ref_logp[i]
            value, d = {"k1": (u, 1.0), "k2": (u * u / 2, u), "k3": (np.expm1(-u) + u, -np.expm1(-u))}[kl]
            row[i] += kl_coef * value
            slope[i] += kl_coef * d
        row[i] *= w
        slope[i] *= w
    return row, slope


def policy_f64(H, W, y, advantages, old_logp=None, ref_logp=None, weights=None, *, temperature=1.0,
               ignore_index=IGNORE_INDEX, reduction=MEAN, n_valid_override=-1, grad_loss=1.0, **kw):
    """loss, logp, row_loss, dH, dW and the gradients' bulks."""
    _, logq, _ = _head(H, W, temperature)
    told = _given(y, W.shape[0], ignore_index)
    logp = np.where(told, logq[np.arange(len(y)), np.where(told, y, 0)], 0.0)
    row, slope = policy_rows_f64(logp, told, advantages, old_logp, ref_logp, weights, **kw)
    w = _weight(int(told.sum()), reduction, n_valid_override)
    grads = head_gradients_f64(H, W, y, slope * w * grad_loss, temperature=temperature, ignore_index=ignore_index)
    return dict(grads, loss=row.sum() * w, logp=logp, row_loss=row)


def preference_pairs_f64(seq_logp, ref_logp=None, *, kind="sigmoid", beta=0.1, label_smoothing=0.0, margin=0.0):
    """pair_loss [P] and its derivative by the pair's difference delta."""
    ratio = seq_logp if ref_logp is None else seq_logp - ref_logp
    delta = ratio[0::2] - ratio[1::2]
    x = beta * delta - margin
    e = label_smoothing
    if kind == "sigmoid":
        loss = (1 - e) * np.logaddexp(0.0, -x) + e * np.logaddexp(0.0, x)
        slope = beta * (e / (1 + np.exp(-x)) - (1 - e) / (1 + np.exp(x)))
    elif kind == "hinge":
        loss, slope = np.maximum(0.0, 1.0 - x), np.where(x < 1.0, -beta, 0.0)
    else:
        loss, slope = (delta - 0.5 / beta) ** 2, 2.0 * (delta - 0.5 / beta)
    return loss, slope


def preference_f64(H, W, y, cu, ref_logp=None, *, temperature=1.0, average=False, ignore_index=IGNORE_INDEX,
                   reduction=MEAN, n_valid_override=-1, grad_loss=1.0, **kw):
    """loss, pair_loss, seq_logp, dH, dW, the gradients' bulks and each row's derivative a."""
    _, logq, _ = _head(H, W, temperature)
    told = _given(y, W.shape[0], ignore_index)
    logp = np.where(told, logq[np.arange(len(y)), np.where(told, y, 0)], 0.0)
    S = len(cu) - 1
    seq, per = np.zeros(S), np.zeros(S)
    for s in range(S):
        rows = slice(cu[s], cu[s + 1])
        n = int(told[rows].sum())
        per[s] = (1.0 / n if n else 0.0) if average else 1.0
        seq[s] = logp[rows][told[rows]].sum() * per[s]
    loss, slope = preference_pairs_f64(seq, ref_logp, **kw)
    w = _weight(S // 2, reduction, n_valid_override)
    a = np.zeros(len(y))
    for s in range(S):
        a[cu[s]:cu[s + 1]] = (slope[s // 2] if s % 2 == 0 else -slope[s // 2]) * per[s] * w * grad_loss
    grads = head_gradients_f64(H, W, y, a, temperature=temperature, ignore_index=ignore_index)
    return dict(grads, loss=loss.sum() * w, pair_loss=loss, seq_logp=seq, a=np.where(told, a, 0.0))


def layernorm_f64(x, w=None, b=None, eps=1e-5):
    """H (not rounded), mean, rstd."""
    mean = x.mean(axis=1)
    var = ((x - mean[:, None]) ** 2).mean(axis=1)
    rstd = 1.0 / np.sqrt(var + eps)
    H = (x - mean[:, None]) * rstd[:, None]
    return {"H": H * (1.0 if w is None else w) + (0.0 if b is None else b), "mean": mean, "rstd": rstd}


def layernorm_backward_f64(x, w, dH, eps=1e-5):
    """dx, dw, db, and the sums of the absolute terms of each."""
    f = layernorm_f64(x, None, None, eps)
    xh, r, d = f["H"], f["rstd"][:, None], x.shape[1]
    g = dH * (1.0 if w is None else w)
    c = (g * xh).sum(axis=1, keepdims=True) / d
    dx = r * (g - g.sum(axis=1, keepdims=True) / d - xh * c)
    bulk = r * (np.abs(g) + np.abs(g).sum(axis=1, keepdims=True) / d +
                np.abs(xh) * np.abs(g * xh).sum(axis=1, keepdims=True) / d)
    return {"dx": dx, "dw": (dH * xh).sum(axis=0), "db": dH.sum(axis=0), "dx_bulk": bulk,
            "dw_bulk": np.abs(dH * xh).sum(axis=0), "db_bulk": np.abs(dH).sum(axis=0)}
