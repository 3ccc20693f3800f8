"""The policy and preference losses and the layer norm on the GPU against the fp64 oracle.

H and W lie on the grid of test_tokens_gpu.py, so their logits are exact in fp32.

Tolerances, with t = tol_lse of test_tokens_gpu.py (the error of lse and of z / T),
eps = 2^-24 and u = 2^-8:
  logp       2 t
  row_loss   r = exp(l - old): l - old rounds eps (|l| + |old|), exp 2^-22, so r errs
             by e_r = 2 t + eps (|l| + |old|) + 2^-21 relative, the clipped side by its
             own roundings (2^-22); KL errs by |dKL| (2 t + eps (|l| + |ref|)) + 2^-21
             (|KL| + |u| + exp(-u)); the sum of both and the weight round 2^-22 of each
             term. Nothing lies within 1e-2 of a border of the clipping range.
  a          |r A| (e_r + 2^-21), and for the KL term the same with its second
             derivative, at most 1 + |dKL|; a rounds once more. The errors of a move
             all of a row's entries alike: their sum over the row's terms, (hot + p) da
             / T, is the slack of the gradients.
  seq_logp   the sum of its tokens' 2 t, eps |S| for the result
  pair_loss  with td = that of both sequences + eps (|ref| of both) the error of delta:
             |slope| td (+ td^2 for ipo) + 2^-22 |loss|
  gradients  each entry of G is rounded to bf16 once (u) behind factors that err by less
             than 2^-10; dW's other operand bf16(scale H) is rounded as well: (2 u + u^2
             + 2^-10) bulk; dH (u + 2^-10) bulk and its own rounding; whole tensors 5e-3.
             From exp tiles (large calls) an entry is rounded (u) and its row's scale
             times rest / bf16(rest), which makes up for the rounding of the label's
             entry -bf16(rest) and is itself off 1 by at most u: (1 + u)^2 - 1 = 2 u + u^2
             for dH, with bf16(scale H) (1 + u)^3 - 1 = 3 u + 3 u^2 + u^3 for dW
  loss       the rows' (pairs') bounds summed, and eps |loss|
  layer norm a sum of d terms in fp32 over lanes and five shuffles errs by g = (d / 32 +
             16) eps of its absolute terms: the mean by em = g mean|x|, the variance by 2
             g + (em rstd)^2 relative, xh by ex = rstd em + |xh| (2 g + (em rstd)^2 +
             2^-21), H by |w| ex + 2^-21 (|xh w| + |b|) and its rounding; dx by (3 g +
             2^-20) of its absolute terms, plus what ex adds to the sum over g xh and to
             its factor, and its rounding; dw by sum |dH| ex + (N eps + 2^-21) sum |dH xh|,
             db by (N eps + 2^-21) sum |dH|
"""
import os
import subprocess
import sys

import numpy as np
import pytest

import oracle
from test_tokens_gpu import U, close, dev, heads, make, np64, tol_lse

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


def _torch():
    import torch
    return torch


def f32(x):
    return np.asarray(x, dtype=np.float32)


def head(H, W, y, T):
    """logp (0 where none is given), which are given, tolerance of logp."""
    z = H @ W.T / T
    lse = np.log(np.exp(z - z.max(axis=1, keepdims=True)).sum(axis=1)) + z.max(axis=1)
    told = (y >= 0) & (y < W.shape[0])
    logp = np.where(told, z[np.arange(len(y)), np.where(told, y, 0)] - lse, 0.0)
    return logp, told, 2 * tol_lse(H, W, lse, T)


def uses_exp_tiles(N, V, chunk):
    rows = min(N, chunk or N)
    return V >= 98304 or rows * V >= (4_500_000 if rows <= 96 else 8_000_000)


def check_gradients(dH, dW, ref, slack, exp=False):
    for got, name in ((dH, "dH"), (dW, "dW")):
        if got is None:
            continue
        rounding = (1 + U) ** ((1 if name == "dH" else 2) + (1 if exp else 0)) - 1
        out = U * np.abs(ref[name]) if got.dtype == _torch().bfloat16 else 0.0
        close(got, ref[name], (rounding + 2.0 ** -10) * ref[name + "_bulk"] + slack[name + "_bulk"] + out + 1e-30, name)
        norm = np.linalg.norm(ref[name])
        assert np.linalg.norm(np64(got) - ref[name]) <= 5e-3 * norm + np.linalg.norm(slack[name + "_bulk"]), name


# --------------------------------------------------------------------------- policy
def policy_inputs(rng, H, W, y, T, kl="k3", old=True, weights=True, clip=(0.2, 0.28), dual=0.0):
    N = len(y)
    logp, told, _ = head(H, W, y, T)
    A = f32(rng.standard_normal(N))
    A[rng.random(N) < 0.05] = 0.0
    step = 0.4 * rng.standard_normal(N)
    for border in (1 - clip[0], 1 + clip[1], max(dual, 1e-3)):
        near = np.abs(step - np.log(border)) < 1e-2
        step = np.where(near, np.log(border) + 1.5e-2, step)
    junk = np.where(told, 0.0, np.nan)   # what lies in masked places is not read
    w = f32(rng.random(N) * (rng.random(N) > 0.1)) if weights else None
    return dict(advantages=f32(A + junk), old_logp=f32(logp - step + junk) if old else None,
                ref_logp=f32(logp - 0.5 * rng.standard_normal(N) + junk) if kl != "none" else None, weights=w)


def call_policy(lce, Ht, Wt, yt, inp, grad=True, **kw):
    args = [None if inp[k] is None else dev(inp[k]) for k in ("advantages", "old_logp", "ref_logp", "weights")]
    if grad:
        return lce.lce_policy_fwd_bwd(Ht, Wt, yt, *args[:3], weights=args[3], **kw)
    return lce.lce_policy_forward(Ht, Wt, yt, *args[:3], weights=args[3], **kw)


def check_policy(outs, H, W, y, inp, *, T=1.0, ignore=-100, chunk=0, **kw):
    """One call's outputs, or a list of such, against the oracle."""
    reduction = dict(mean=oracle.MEAN, sum=1)[kw.pop("reduction", "mean")]
    args = [None if inp[k] is None else np.nan_to_num(inp[k].astype(np.float64)) for k in
            ("advantages", "old_logp", "ref_logp", "weights")]
    ref = oracle.policy_f64(H, W, y, *args, temperature=T, ignore_index=ignore, reduction=reduction, **kw)
    scale_kw = {k: kw[k] for k in ("n_valid_override", "grad_loss") if k in kw}
    logp, told, tol = head(H, W, np.where(y == ignore, -1, y), T)
    A, old, rl, w = args
    w = np.ones(len(y)) if w is None else w
    r = np.ones(len(y)) if old is None else np.exp(logp - old)
    e_r = tol + (0 if old is None else EPS * (np.abs(logp) + np.abs(old))) + 2.0 ** -21
    side = np.maximum(np.abs(r * A), 4 * np.abs(A))
    row_tol = side * (e_r + 2.0 ** -20)
    a_tol = np.abs(r * A) * (e_r + 2.0 ** -20)
    kl, beta = kw.get("kl", "none"), abs(kw.get("kl_coef", 0.0))
    if kl != "none":
        u = logp - rl
        value, d = {"k1": (u, 1.0 + 0 * u), "k2": (u * u / 2, u), "k3": (np.expm1(-u) + u, -np.expm1(-u))}[kl]
        e_u = tol + EPS * (np.abs(logp) + np.abs(rl))
        row_tol = row_tol + beta * (np.abs(d) * e_u + e_u ** 2 + 2.0 ** -20 * (np.abs(value) + np.abs(u) + np.exp(-u)))
        a_tol = a_tol + beta * ((1 + np.abs(d)) * e_u + 2.0 ** -20 * (1 + np.abs(d)))
    row_tol, a_tol = np.where(told, row_tol * np.abs(w), 0.0), np.where(told, a_tol * np.abs(w), 0.0)
    n = kw.get("n_valid_override", -1)
    weight = 1.0 if reduction == 1 else 1.0 / max(n if n >= 0 else int(told.sum()), 1)
    if n == 0 and reduction != 1:
        weight = 0.0
    slack = oracle.head_gradients_f64(H, W, y, a_tol * weight * abs(scale_kw.get("grad_loss", 1.0)), temperature=T,
                                      ignore_index=ignore)
    for out in outs if isinstance(outs, list) else [outs]:
        loss, got_logp, row = out[:3]
        close(got_logp, ref["logp"], np.where(told, tol, 0.0), "logp")
        close(row, ref["row_loss"], row_tol + 2.0 ** -22 * np.abs(ref["row_loss"]), "row_loss")
        close(loss, np.array([ref["loss"]]), row_tol.sum() * weight + 2 * EPS * (abs(ref["loss"]) + np.abs(ref["row_loss"]).sum() * weight) + 1e-30,
              "loss")
        if len(out) == 5:
            check_gradients(out[3], out[4], ref, slack, uses_exp_tiles(len(y), W.shape[0], chunk))
    return ref


# N, d, V, T, chunk, kl, old, weights, dual
POLICY_CASES = [
    (1, 8, 1, 1.0, 0, "none", True, False, 0.0),       # one word: its probability is 1, nothing to learn
    (1, 64, 37, 1.0, 0, "k3", True, True, 0.0),
    (3, 72, 2, 0.7, 0, "k1", False, False, 0.0),
    (5, 64, 128, 2.0, 0, "k2", True, True, 1.5),
    (33, 136, 129, 1.0, 0, "k3", True, False, 3.0),    # one column in the second half tile
    (64, 256, 4096, 1.0, 0, "none", False, True, 0.0),
    (96, 64, 4099, 0.5, 0, "k3", True, True, 0.0),
    (97, 64, 4099, 1.3, 0, "k2", True, False, 2.0),    # past the few-rows kernel
    (129, 136, 5003, 1.0, 64, "k3", True, True, 0.0),  # three chunks, the last of one row
    (300, 256, 3001, 1.0, 256, "k1", True, True, 1.2),
    (513, 264, 1000, 0.9, 200, "none", True, False, 0.0),
    (700, 128, 20011, 1.0, 0, "k3", True, True, 3.0),
    (1000, 512, 9000, 1.0, 0, "k3", False, True, 0.0),
    # enough logits for exp tiles
    (97, 64, 250007, 1.0, 0, "k3", True, True, 0.0),
    (300, 136, 80101, 0.8, 0, "k2", True, True, 3.0),
    (501, 64, 100003, 1.0, 250, "k3", True, False, 0.0),   # three chunks, the last of one row
    (400, 64, 65537, 1.0, 0, "none", False, True, 0.0),
    (300, 64, 80101, 0.1, 0, "k3", True, True, 0.0),       # labels far below the largest logit: exact tiles
    (501, 64, 100003, 0.1, 250, "k2", True, True, 0.0),    # the same in three chunks
    (6200, 64, 7301, 1.0, 0, "k3", True, True, 3.0),       # exp tiles of two launches, one backward
    (6200, 64, 7301, 0.1, 0, "none", True, False, 0.0),    # the same by exact tiles
]


@pytest.mark.parametrize("N,d,V,T,chunk,kl,old,weights,dual", POLICY_CASES)
def test_policy(cuda_lib, N, d, V, T, chunk, kl, old, weights, dual):
    torch = _torch()
    rng, H, W, y = make(N, d, V, seed=N + V)
    Ht, Wt = heads(H, W)
    inp = policy_inputs(rng, H, W, y, T, kl, old, weights, dual=dual)
    kw = dict(clip_low=0.2, clip_high=0.28, dual_clip=dual, kl=kl, kl_coef=0.0 if kl == "none" else 0.3)
    outs = [call_policy(cuda_lib, Ht, Wt, dev(y), inp, temperature=T, chunk_tokens=chunk, dW_dtype=dt, sync_check=True, **kw)
            for dt in (torch.float32, torch.bfloat16)]
    out = outs[-1]
    outs.append(call_policy(cuda_lib, Ht, Wt, dev(y), inp, grad=False, temperature=T, chunk_tokens=chunk, sync_check=True, **kw))
    check_policy(outs, H, W, y, inp, T=T, chunk=chunk, **kw)
    again = call_policy(cuda_lib, Ht, Wt, dev(y), inp, temperature=T, chunk_tokens=chunk, dW_dtype=torch.bfloat16, **kw)
    for a, b in zip(out, again):
        assert torch.equal(a, b)


def test_policy_sum_override_accumulation_and_frozen_sides(cuda_lib):
    torch = _torch()
    rng, H, W, y = make(150, 64, 700)
    Ht, Wt = heads(H, W)
    inp = policy_inputs(rng, H, W, y, 1.0)
    kw = dict(kl="k3", kl_coef=0.1, clip_low=0.2, clip_high=0.28)
    for more in (dict(reduction="sum"), dict(n_valid_override=1000), dict(n_valid_override=0)):
        for chunk in (0, 64):
            out = call_policy(cuda_lib, Ht, Wt, dev(y), inp, chunk_tokens=chunk, **kw, **more)
            check_policy(out, H, W, y, inp, **kw, **more)
    g = torch.tensor([-2.5], device="cuda")
    for chunk in (0, 64):
        out = call_policy(cuda_lib, Ht, Wt, dev(y), inp, grad_loss=g, chunk_tokens=chunk, **kw)
        check_policy(out, H, W, y, inp, grad_loss=-2.5, **kw)
        base = torch.randn(700, 64, device="cuda")
        dW = base.clone()
        acc = call_policy(cuda_lib, Ht, Wt, dev(y), inp, grad_loss=g, dW=dW, accumulate_dW=True, chunk_tokens=chunk, **kw)
        assert acc[4] is dW and (dW - base - out[4]).abs().max() <= 2.0 ** -22 * (base.abs().max() + out[4].abs().max())
        only_dH = call_policy(cuda_lib, Ht, Wt, dev(y), inp, grad_loss=g, need_dW=False, chunk_tokens=chunk, **kw)
        only_dW = call_policy(cuda_lib, Ht, Wt, dev(y), inp, grad_loss=g, need_dH=False, chunk_tokens=chunk, **kw)
        assert only_dH[4] is None and torch.equal(only_dH[3], out[3])
        assert only_dW[3] is None and torch.equal(only_dW[4], out[4])


@pytest.mark.parametrize("N", [40, 300])
def test_policy_masked_weightless_and_clipped_rows(cuda_lib, N):
    """Rows without a token or with a weight of 0 may hold NaN; clipped rows have a zero gradient; no row at all."""
    torch = _torch()
    rng, H, W, y = make(N, 64, 900)
    inp = policy_inputs(rng, H, W, y, 1.0, "none")
    inp["weights"] = f32(np.ones(N))
    inp["weights"][3:9] = 0.0
    y[3:9] = 5
    Ht, Wt = heads(H, W)
    clean = call_policy(cuda_lib, Ht, Wt, dev(y), inp)
    bad = Ht.clone()
    bad[torch.from_numpy(y < 0).cuda()] = float("nan")
    bad[3:9] = float("nan")
    bad[5] = float("inf")
    got = call_policy(cuda_lib, bad, Wt, dev(y), inp, sync_check=True)
    keep = np.ones(N, bool)
    keep[3:9] = False
    for k in (0, 2, 3, 4):
        assert torch.equal(got[k], clean[k]), k
    assert torch.equal(got[1][torch.from_numpy(keep).cuda()], clean[1][torch.from_numpy(keep).cuda()])
    assert not got[3][3:9].any() and not got[2][3:9].any()
    # every positive advantage clipped from above: nothing to learn from it
    logp, told, _ = head(H, W, y, 1.0)
    inp = dict(advantages=f32(np.ones(N)), old_logp=f32(logp - 1.0), ref_logp=None, weights=None)
    loss, _, row, dH, dW = call_policy(cuda_lib, Ht, Wt, dev(y), inp)
    assert not dH.any() and not dW.any() and (row.cpu().numpy()[told] == np.float32(-1.2)).all()
    # no token given
    none = np.full(N, -100)
    for chunk in (0, 16):
        out = call_policy(cuda_lib, torch.full_like(Ht, float("nan")), Wt, dev(none), inp, chunk_tokens=chunk)
        assert all(not x.any() for x in out)


def test_policy_extreme_ratios(cuda_lib):
    """A ratio that overflows: no share without an advantage, clipped with a positive one, bounded by the dual clip."""
    torch = _torch()
    _, H, W, y = make(8, 64, 300)
    y[:] = np.arange(8)
    Ht, Wt = heads(H, W)
    A = f32([0.0, 1.0, -1.0, -1.0, 0.0, 1.0, 2.0, -2.0])
    old = f32([-500.0, -500.0, -500.0, -1.0, 500.0, 500.0, 500.0, 500.0])
    inp = dict(advantages=A, old_logp=old, ref_logp=None, weights=None)
    loss, logp, row, dH, dW = call_policy(cuda_lib, Ht, Wt, dev(y), inp, dual_clip=3.0)
    assert torch.isfinite(dH).all() and torch.isfinite(dW).all()
    row = row.cpu().numpy()
    assert row[0] == 0 and row[1] == np.float32(-1.2) and row[2] == 3.0 and row[4] == 0
    assert row[5] == 0.0 and row[6] == 0.0                     # r = 0 of a positive advantage: min(0, 0.8 A)
    np.testing.assert_allclose(row[7], 1.6, rtol=1e-6)         # r = 0 of a negative one: clipped from below
    zero = dH.cpu().float().numpy()
    assert not zero[[0, 1, 2, 4, 5, 6, 7]].any()
    infinite = call_policy(cuda_lib, Ht, Wt, dev(y), dict(inp, advantages=f32(-np.ones(8))))
    assert np.isinf(infinite[2].cpu().numpy()[:3]).all()       # without it the loss is what the formula says


def test_policy_labels_out_of_range(cuda_lib):
    torch = _torch()
    rng, H, W, y = make(130, 64, 500)
    inp = policy_inputs(rng, H, W, y, 1.0)
    Ht, Wt = heads(H, W)
    wrong = y.copy()
    wrong[[2, 77]] = [500, -7]
    masked = y.copy()
    masked[[2, 77]] = -100
    for chunk in (0, 32):
        for grad in (True, False):
            got = call_policy(cuda_lib, Ht, Wt, dev(wrong), inp, grad=grad, kl="k3", kl_coef=0.1, chunk_tokens=chunk)
            want = call_policy(cuda_lib, Ht, Wt, dev(masked), inp, grad=grad, kl="k3", kl_coef=0.1, chunk_tokens=chunk)
            for a, b in zip(got, want):
                assert torch.equal(a, b)
            with pytest.raises(cuda_lib.LCEError) as err:
                call_policy(cuda_lib, Ht, Wt, dev(wrong), inp, grad=grad, chunk_tokens=chunk, sync_check=True)
            assert err.value.code == cuda_lib.LCE_ERR_LABEL_RANGE
    # an ignore_index inside the vocabulary
    y = np.abs(y) % 500
    kw = dict(kl="k3", kl_coef=0.1, clip_low=0.2, clip_high=0.28)
    inp = policy_inputs(rng, H, W, np.where(y == 7, -1, y), 1.0)
    y[5:9] = 7
    for k in ("advantages", "old_logp", "ref_logp"):
        inp[k] = np.nan_to_num(inp[k])
    out = call_policy(cuda_lib, Ht, Wt, dev(y), inp, ignore_index=7, **kw)
    check_policy(out, H, W, y, inp, ignore=7, **kw)


# --------------------------------------------------------------------------- preference
def bounds(rng, N, pairs, front=0, back=0, empty=()):
    cut = np.sort(rng.integers(front, N - back + 1, 2 * pairs - 1)) if pairs else np.array([], dtype=np.int64)
    cu = np.concatenate([[front], cut, [N - back]]) if pairs else np.array([front])
    for s in empty:
        cu[s + 1] = cu[s]
        cu = np.maximum.accumulate(cu)
    return cu.astype(np.int64)


def call_preference(lce, Ht, Wt, y, cu, ref, grad=True, **kw):
    r = None if ref is None else dev(f32(ref))
    if grad:
        return lce.lce_preference_fwd_bwd(Ht, Wt, dev(y), dev(cu), r, **kw)
    return lce.lce_preference_forward(Ht, Wt, dev(y), dev(cu), r, **kw)


def check_preference(outs, H, W, y, cu, ref_logp, *, T=1.0, average=False, chunk=0, **kw):
    """One call's outputs, or a list of such, against the oracle."""
    reduction = dict(mean=oracle.MEAN, sum=1)[kw.pop("reduction", "mean")]
    rl = None if ref_logp is None else f32(ref_logp).astype(np.float64)
    ref = oracle.preference_f64(H, W, y, cu, rl, temperature=T, average=average, reduction=reduction, **kw)
    logp, told, tol = head(H, W, y, T)
    S = len(cu) - 1
    ts, per = np.zeros(S), np.ones(S)
    for s in range(S):
        rows = np.arange(cu[s], cu[s + 1])
        rows = rows[told[rows]]
        per[s] = 1.0 / max(len(rows), 1) if average else 1.0
        ts[s] = tol[rows].sum() * per[s]
    td = ts[0::2] + ts[1::2] + (0 if rl is None else EPS * (np.abs(rl[0::2]) + np.abs(rl[1::2])))
    beta = float(np.float32(kw.get("beta", 0.1)))
    kind = kw.get("kind", "sigmoid")
    _, slope = oracle.preference_pairs_f64(ref["seq_logp"], rl, **{k: kw[k] for k in
                                           ("kind", "beta", "label_smoothing", "margin") if k in kw})
    # beta, margin and label_smoothing arrive in fp32: relative eps each, of beta |delta|, margin and the loss
    ratio = ref["seq_logp"] if rl is None else ref["seq_logp"] - rl
    delta = np.abs(ratio[0::2] - ratio[1::2])
    tx = beta * td + 2 * EPS * (beta * delta + abs(kw.get("margin", 0.0)))
    if kind == "ipo":
        pair_tol = np.abs(slope) * (td + EPS / beta) + (td + EPS / beta) ** 2
        slope_tol = 2 * (td + EPS / beta)
    else:
        pair_tol = tx * (1.0 if kind == "hinge" else np.minimum(1.0, np.abs(slope) / beta + tx)) + 2 * EPS * (1 + beta * delta)
        slope_tol = 0 * td if kind == "hinge" else beta * np.minimum(1.0, np.abs(slope) / beta + tx) * tx + 4 * EPS * beta
    n = kw.get("n_valid_override", -1)
    n = n if n >= 0 else S // 2
    weight = 1.0 if reduction == 1 else (1.0 / n if n else 0.0)
    a = np.zeros(len(y))
    for s in range(S):
        a[cu[s]:cu[s + 1]] = (slope_tol[s // 2] + 2.0 ** -22 * abs(slope[s // 2])) * per[s] * weight
    a = np.where(told, a, 0.0) * abs(kw.get("grad_loss", 1.0))
    slack = oracle.head_gradients_f64(H, W, y, a, temperature=T)
    outside = np.ones(len(y), bool)
    outside[cu[0]:cu[-1]] = False
    for out in outs if isinstance(outs, list) else [outs]:
        close(out[2], ref["seq_logp"], ts + 2 * EPS * np.abs(ref["seq_logp"]), "seq_logp")
        close(out[1], ref["pair_loss"], pair_tol + 2.0 ** -22 * np.abs(ref["pair_loss"]), "pair_loss")
        close(out[0], np.array([ref["loss"]]), (pair_tol.sum() + 2.0 ** -22 * np.abs(ref["pair_loss"]).sum()) * weight + 1e-30, "loss")
        if len(out) == 5:
            check_gradients(out[3], out[4], ref, slack, uses_exp_tiles(len(y), W.shape[0], chunk))
            if out[3] is not None:
                assert not np64(out[3])[outside | ~told].any()
    return ref


# N, d, V, pairs, T, chunk, kind, average, ref
PREFERENCE_CASES = [
    (2, 8, 1, 1, 1.0, 0, "sigmoid", False, False),
    (2, 64, 37, 1, 1.0, 0, "sigmoid", False, True),
    (7, 72, 129, 1, 0.7, 0, "hinge", True, True),
    (40, 64, 900, 3, 1.0, 0, "ipo", False, True),
    (96, 64, 4099, 5, 1.0, 0, "sigmoid", True, False),
    (97, 64, 4099, 5, 1.0, 0, "sigmoid", False, True),
    (130, 136, 5003, 4, 1.0, 64, "sigmoid", False, True),   # three chunks: the logits are computed twice
    (300, 256, 3001, 2, 1.0, 128, "ipo", True, True),
    (513, 264, 1000, 20, 0.9, 200, "hinge", False, True),
    (700, 128, 20011, 3, 1.0, 0, "sigmoid", False, True),
    (600, 64, 700, 290, 1.0, 0, "sigmoid", False, True),    # sequences of a token or none
    # enough logits for exp tiles
    (97, 64, 250007, 2, 1.0, 0, "sigmoid", False, True),
    (300, 136, 80101, 4, 0.8, 0, "ipo", True, True),
    (501, 64, 100003, 3, 1.0, 250, "hinge", False, True),   # three chunks: the logits are computed twice
    (6200, 64, 7301, 5, 1.0, 0, "sigmoid", True, False),    # exp tiles of two launches, kept for one backward
    (300, 64, 80101, 3, 0.1, 0, "sigmoid", True, True),     # labels far below the largest logit: exact tiles
    (300, 64, 80101, 30, 0.1, 0, "hinge", True, True),      # the same with more pairs than the rows' launch takes
    (6200, 64, 7301, 5, 0.1, 0, "sigmoid", True, True),     # exact tiles of two launches
]


@pytest.mark.parametrize("N,d,V,pairs,T,chunk,kind,average,ref", PREFERENCE_CASES)
def test_preference(cuda_lib, N, d, V, pairs, T, chunk, kind, average, ref):
    torch = _torch()
    rng, H, W, y = make(N, d, V, seed=N + V)
    Ht, Wt = heads(H, W)
    cu = bounds(rng, N, pairs, *((1, 3, (2,)) if N >= 40 else ()))
    beta = 1.5 if average else 0.1
    kw = dict(kind=kind, beta=beta, margin=0.0 if kind == "ipo" else 0.25, average=average,
              label_smoothing=0.1 if kind == "sigmoid" else 0.0)
    rl = None
    if ref:
        seq = oracle.preference_f64(H, W, y, cu, None, temperature=T, average=average, kind=kind, beta=beta)["seq_logp"]
        x = 0.25 + rng.standard_normal(pairs) * 1.5
        x = np.where(np.abs(x - 0.25 - 1.0) < 0.05, 1.4, x)      # away from the hinge's corner
        rl = f32(seq + rng.standard_normal(2 * pairs))
        rl[0::2] = (seq[0::2] - seq[1::2]) + rl[1::2].astype(np.float64) - x / beta
    narrow = cu.astype(np.int32)
    outs = [call_preference(cuda_lib, Ht, Wt, y, c, rl, temperature=T, chunk_tokens=chunk, dW_dtype=dt, sync_check=True, **kw)
            for dt, c in ((torch.float32, narrow), (torch.bfloat16, cu))]
    out = outs[-1]
    outs.append(call_preference(cuda_lib, Ht, Wt, y, narrow, rl, grad=False, temperature=T, chunk_tokens=chunk, sync_check=True, **kw))
    check_preference(outs, H, W, y, cu, rl, T=T, chunk=chunk, **kw)
    again = call_preference(cuda_lib, Ht, Wt, y, narrow, rl, temperature=T, chunk_tokens=chunk, dW_dtype=torch.bfloat16, **kw)
    for a, b in zip(out, again):
        assert torch.equal(a, b)


def test_preference_sum_override_accumulation_and_frozen_sides(cuda_lib):
    torch = _torch()
    rng, H, W, y = make(150, 64, 700)
    Ht, Wt = heads(H, W)
    cu = bounds(rng, 150, 4, 0, 10)
    for more in (dict(reduction="sum"), dict(n_valid_override=100), dict(n_valid_override=0)):
        for chunk in (0, 64):
            check_preference(call_preference(cuda_lib, Ht, Wt, y, cu, None, chunk_tokens=chunk, **more), H, W, y, cu, None, **more)
    g = torch.tensor([3.5], device="cuda")
    for chunk in (0, 64):
        out = call_preference(cuda_lib, Ht, Wt, y, cu, None, grad_loss=g, chunk_tokens=chunk)
        check_preference(out, H, W, y, cu, None, grad_loss=3.5)
        base = torch.randn(700, 64, device="cuda")
        dW = base.clone()
        call_preference(cuda_lib, Ht, Wt, y, cu, None, grad_loss=g, dW=dW, accumulate_dW=True, chunk_tokens=chunk)
        assert (dW - base - out[4]).abs().max() <= 2.0 ** -22 * (base.abs().max() + out[4].abs().max())
        only_dH = call_preference(cuda_lib, Ht, Wt, y, cu, None, grad_loss=g, need_dW=False, chunk_tokens=chunk)
        only_dW = call_preference(cuda_lib, Ht, Wt, y, cu, None, grad_loss=g, need_dH=False, chunk_tokens=chunk)
        assert only_dH[4] is None and torch.equal(only_dH[3], out[3])
        assert only_dW[3] is None and torch.equal(only_dW[4], out[4])


@pytest.mark.parametrize("N", [60, 300])
def test_preference_rows_outside_may_hold_nan(cuda_lib, N):
    """Padding, prompts and rows in no sequence may hold anything."""
    torch = _torch()
    rng, H, W, y = make(N, 64, 900)
    cu = bounds(rng, N, 3, 4, 9)
    Ht, Wt = heads(H, W)
    for chunk in (0, 32):
        clean = call_preference(cuda_lib, Ht, Wt, y, cu, None, chunk_tokens=chunk)
        bad = Ht.clone()
        bad[:4] = float("nan")
        bad[N - 9:] = float("nan")
        bad[torch.from_numpy(y < 0).cuda()] = float("inf")
        got = call_preference(cuda_lib, bad, Wt, y, cu, None, chunk_tokens=chunk, sync_check=True)
        for a, b in zip(got, clean):
            assert torch.equal(a, b)


def test_preference_bad_bounds_no_pairs_and_no_rows(cuda_lib):
    """Bounds that fall or leave the rows are reported, their pairs left out."""
    torch = _torch()
    rng, H, W, y = make(100, 64, 300)
    Ht, Wt = heads(H, W)
    good = np.array([0, 20, 40, 60, 80, 90, 100])
    want = {c: call_preference(cuda_lib, Ht, Wt, y, good, None, reduction="sum", chunk_tokens=c) for c in (0, 32)}
    for wrong, pair in ((101, 2), (2 ** 40, 2), (-3, 0)):
        cu = good.copy()
        cu[6 if pair == 2 else 0] = wrong
        for chunk in (0, 32):
            out = call_preference(cuda_lib, Ht, Wt, y, cu, None, reduction="sum", chunk_tokens=chunk)
            assert out[1][pair] == 0 and not out[3][good[2 * pair]:good[2 * pair + 2]].any()
            others = [k for k in range(3) if k != pair]
            assert torch.equal(out[1][others], want[chunk][1][others])
            with pytest.raises(cuda_lib.LCEError) as err:
                call_preference(cuda_lib, Ht, Wt, y, cu, None, chunk_tokens=chunk, sync_check=True)
            assert err.value.code == cuda_lib.LCE_ERR_LABEL_RANGE
    fall = good.copy()
    fall[3] = 30
    with pytest.raises(cuda_lib.LCEError) as err:
        call_preference(cuda_lib, Ht, Wt, y, fall, None, grad=False, sync_check=True)
    assert err.value.code == cuda_lib.LCE_ERR_LABEL_RANGE
    for cu in (np.array([0]), np.array([30])):
        for chunk in (0, 32):
            out = call_preference(cuda_lib, Ht, Wt, y, cu, None, chunk_tokens=chunk, sync_check=True)
            assert out[1].shape == (0,) and all(not x.any() for x in out)
    for dt in (torch.float32, torch.bfloat16):
        out = call_preference(cuda_lib, Ht[:0], Wt, y[:0], np.zeros(5, np.int64), None, dW_dtype=dt, sync_check=True)
        np.testing.assert_allclose(out[0].item(), np.log(2.0), rtol=1e-7)
        assert out[3].shape == (0, 64) and not out[4].any() and not out[2].any()
        inp = dict(advantages=f32([]), old_logp=None, ref_logp=None, weights=None)
        out = call_policy(cuda_lib, Ht[:0], Wt, dev(y[:0]), inp, dW_dtype=dt, sync_check=True)
        assert out[0].item() == 0 and out[3].shape == (0, 64) and not out[4].any()


@pytest.mark.parametrize("N", [40, 300])
def test_preference_without_pairs_needs_no_bounds(cuda_lib, N):
    """The C call with pairs = 0 and no pointers of pairs: loss 0, gradients 0 (kept logits, exp tiles, two chunks)."""
    import ctypes
    torch = _torch()
    V, d = 80101, 64
    _, H, W, y = make(N, d, V)
    Ht, Wt, yt = *heads(H, W), dev(y)
    lib, p = cuda_lib.load(), lambda t: ctypes.c_void_p(t.data_ptr())
    for chunk in (0, 32):
        opts = cuda_lib.make_opts(chunk_tokens=chunk, sync_check=True)
        pref = cuda_lib.LcePreference(0.1, 0.0, 0.0, 0, 0, 0)
        ws = torch.empty(cuda_lib.lce_preference_workspace_size(N, d, V, 0, opts=opts), dtype=torch.uint8, device="cuda")
        loss, dH, dW = torch.ones(1, device="cuda"), torch.ones_like(Ht), torch.ones(V, d, device="cuda")
        rc = lib.lce_preference_fwd_bwd(p(Ht), p(Wt), p(yt), N, d, V, None, 0, 1.0, ctypes.byref(pref), None, None, 0, p(loss),
                                        None, None, p(dH), p(dW), ctypes.byref(opts), p(ws), ws.numel(),
                                        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert rc == 0 and loss.item() == 0 and not dH.any() and not dW.any()


# --------------------------------------------------------------------------- the heads' real sizes
@pytest.mark.parametrize("N,d,V,chunk", [(70, 2048, 151936, 0), (6500, 2048, 151936, 0), (700, 7168, 151655, 512),
                                         (16500, 64, 151655, 0)])
def test_full_heads_sampled(cuda_lib, N, d, V, chunk):
    """Few rows with kept logits, exp tiles of two launches behind one backward, two chunks of the widest head, a tile of
    more than 2^31 entries: rows of both sides of every boundary and vocabulary rows of the tails, against fp64."""
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(N)
    sigma = 0.02 if d <= 2048 else 0.01
    if d == 64:
        sigma = 0.1
    W = (torch.randn(V, d, generator=g, device="cuda") * (sigma * 1024)).round().clamp(-127, 127).div(1024).bfloat16()
    y = torch.randint(0, V, (N,), generator=g, device="cuda")
    H = torch.randn(N, d, generator=g, device="cuda")
    H += W[y].float() * (14.0 * torch.rand(N, 1, generator=g, device="cuda") / (sigma * sigma * d))
    H = (H * 16).round().clamp(-127, 127).div(16).bfloat16()
    y[::17] = oracle.IGNORE_INDEX
    edge = chunk or {70: 35, 6500: 3328, 16500: 4352}[N]
    rows = np.unique([0, 1, edge - 1, edge, edge + 1, N // 3, N - 2, N - 1])
    cols = np.array([0, 127, 128, 255, 256, V // 2, V - 130, V - 2, V - 1])
    Hn, Wn, yn = np64(H), np64(W), y.cpu().numpy()
    lse = torch.cat([torch.logsumexp(H[r:r + 512].double() @ W.double().t(), 1) for r in range(0, N, 512)]).cpu().numpy()
    told = yn >= 0
    logp = np.where(told, (Hn * Wn[np.where(told, yn, 0)]).sum(1) - lse, 0.0)
    p = np.exp(Hn @ Wn[cols].T - lse[:, None])
    hot = (yn[:, None] == cols[None, :]).astype(float)
    exp = uses_exp_tiles(N, V, chunk)
    at = torch.from_numpy(rows).cuda()

    def check(dH, dW, a):   # a: d loss / d logp
        a = np.where(told, a, 0.0)
        part = oracle.head_gradients_f64(Hn[rows], Wn, yn[rows], a[rows])
        none = {"dH_bulk": 2.0 ** -11 * part["dH_bulk"]}          # what logp's error does to a
        check_gradients(dH[at], None, part, none, exp)
        G = (hot - p) * a[:, None]
        size = (hot + p) * np.abs(a)[:, None]
        bulk = size.T @ np.abs(Hn)
        check_gradients(None, dW[torch.from_numpy(cols).cuda()], {"dW": G.T @ Hn, "dW_bulk": bulk}, {"dW_bulk": 2.0 ** -11 * bulk}, exp)

    rng = np.random.default_rng(1)
    A = f32(rng.standard_normal(N))
    old = f32(logp - 0.05)                                        # every ratio inside the range
    loss, got, row, dH, dW = cuda_lib.lce_policy_fwd_bwd(H, W, y, dev(A), dev(old), dW_dtype=torch.bfloat16, chunk_tokens=chunk,
                                                         sync_check=True)
    n = int(told.sum())
    r = np.exp(logp - old)
    close(got, logp, 2.0 ** -14, "logp")
    close(row, np.where(told, -r * A, 0.0), 2.0 ** -12 * np.abs(A) + 1e-30, "row_loss")
    close(loss, np.array([-(r * A)[told].sum() / n]), 2.0 ** -12 * np.abs(A[told]).mean(), "loss")
    check(dH, dW, -r * A / n)
    fwd = cuda_lib.lce_policy_forward(H, W, y, dev(A), dev(old), chunk_tokens=chunk)
    close(fwd[1], logp, 2.0 ** -14, "logp of the forward")
    pairs = 3
    cu = bounds(rng, N, pairs, 0, N // 20)
    out = cuda_lib.lce_preference_fwd_bwd(H, W, y, dev(cu), average=True, beta=2.0, chunk_tokens=chunk, sync_check=True)
    seq = np.array([logp[cu[s]:cu[s + 1]][told[cu[s]:cu[s + 1]]].mean() for s in range(2 * pairs)])
    count = np.array([told[cu[s]:cu[s + 1]].sum() for s in range(2 * pairs)])
    pl, slope = oracle.preference_pairs_f64(seq, beta=2.0)
    close(out[2], seq, 2.0 ** -14, "seq_logp")
    close(out[1], pl, 2.0 ** -11, "pair_loss")
    a = np.zeros(N)
    for s in range(2 * pairs):
        a[cu[s]:cu[s + 1]] = (slope[s // 2] if s % 2 == 0 else -slope[s // 2]) / pairs / count[s]
    check(out[3], out[4], a)


# --------------------------------------------------------------------------- exp tiles
def test_exp_tiles_masked_rows_of_nan(cuda_lib):
    """Masked and weightless rows may hold NaN where exp tiles are used; a given row of NaN has a loss of NaN and leaves
    the other rows' dH alone."""
    torch = _torch()
    N, V = 300, 80101
    rng, H, W, y = make(N, 64, V)
    Ht, Wt = heads(H, W)
    inp = policy_inputs(rng, H, W, y, 1.0, "none")
    masked = torch.from_numpy(y < 0).cuda()
    clean = call_policy(cuda_lib, Ht, Wt, dev(y), inp)
    bad = Ht.clone()
    bad[masked] = float("nan")
    for a, b in zip(call_policy(cuda_lib, bad, Wt, dev(y), inp, sync_check=True), clean):
        assert torch.equal(a, b)
    cu = bounds(rng, N, 3, 4, 9)
    clean = call_preference(cuda_lib, Ht, Wt, y, cu, None)
    for a, b in zip(call_preference(cuda_lib, bad, Wt, y, cu, None, sync_check=True), clean):
        assert torch.equal(a, b)
    # a weight of 0, or no sequence, on a row with a given token: the exact tiles take over
    row = int(np.flatnonzero(y >= 0)[3])
    inp["weights"] = f32(np.ones(N))
    inp["weights"][row] = 0.0
    bad[row] = float("nan")
    got = call_policy(cuda_lib, bad, Wt, dev(y), inp, sync_check=True)
    zero = Ht.clone()
    zero[row] = 0
    want = call_policy(cuda_lib, zero, Wt, dev(y), inp)
    assert got[2][row] == 0 and not got[3][row].any() and torch.isfinite(got[4]).all()
    assert torch.linalg.vector_norm(got[4] - want[4]) <= 5e-3 * torch.linalg.vector_norm(want[4])
    assert torch.linalg.vector_norm((got[3] - want[3]).float()) <= 5e-3 * torch.linalg.vector_norm(want[3].float())
    inp["weights"][row] = 1.0
    got = call_policy(cuda_lib, bad, Wt, dev(y), inp)
    rest = torch.arange(N, device="cuda") != row
    assert got[0].isnan().all() and got[2][row].isnan() and torch.isfinite(got[3][rest]).all() and got[3][row].isnan().all()


def test_exp_tiles_of_a_label_past_fp32(cuda_lib):
    """A label's logit that overflows to infinity, the others finite: NaN, as inf - inf is, in that row alone."""
    torch = _torch()
    N, d, V = 300, 64, 80101
    rng, H, W, y = make(N, d, V, seed=7)
    rows = np.flatnonzero(y >= 0)
    row, label = int(rows[10]), 70000
    y[rows[y[rows] == label]] = 5
    y[row] = label
    W[:, 0] = 0.0
    H[:, 0] = 0.0
    W[label, 0] = 2.0 ** 127
    Ht, Wt = heads(H, W)
    inp = policy_inputs(rng, H, W, y, 1.0, weights=False)
    inp["advantages"][row] = 1.0
    want = call_policy(cuda_lib, Ht, Wt, dev(y), inp)
    cu = bounds(rng, N, 3)
    seq = int(np.searchsorted(cu, row, side="right")) - 1
    want_seq = call_preference(cuda_lib, Ht, Wt, y, cu, None)[2]
    Ht[row, 0] = 2.0 ** 127
    got = call_policy(cuda_lib, Ht, Wt, dev(y), inp, sync_check=True)
    rest = torch.arange(N, device="cuda") != row
    assert got[0].isnan().all() and got[1][row].isnan() and got[2][row].isnan()
    assert ((got[1] - want[1])[rest].abs() <= 2.0 ** -14).all() and torch.isfinite(got[3][rest]).all()
    got = call_preference(cuda_lib, Ht, Wt, y, cu, None, sync_check=True)
    others = torch.arange(6, device="cuda") != seq
    assert got[0].isnan().all() and (0 <= seq < 6) and got[2][seq].isnan() and torch.isfinite(got[2][others]).all()
    assert torch.isfinite(want_seq).all()


@pytest.mark.parametrize("N,V", [(1, 100003), (5, 98304), (60, 80101), (96, 131072)])
def test_exp_tiles_of_few_rows(cuda_lib, N, V):
    """Few rows of a large vocabulary, and the same with a label out of the tile's range."""
    rng, H, W, y = make(N, 64, V, seed=N)
    y[-1] = V - 1
    for far in (False, True):
        if far:
            W[:, 0] = 0.0
            H[:, 0] = 0.0
            W[y[-1], 0] = -1.0
            H[-1, 0] = 100.0
        Ht, Wt = heads(H, W)
        inp = policy_inputs(rng, H, W, y, 1.0)
        kw = dict(clip_low=0.2, clip_high=0.28, kl="k3", kl_coef=0.1)
        check_policy(call_policy(cuda_lib, Ht, Wt, dev(y), inp, sync_check=True, **kw), H, W, y, inp, **kw)
        cu = bounds(rng, N, 2)
        check_preference(call_preference(cuda_lib, Ht, Wt, y, cu, None, average=True, sync_check=True), H, W, y, cu, None,
                         average=True)


@pytest.mark.parametrize("shift", [50.0, 70.0, 200.0])
def test_exp_tiles_of_one_far_label(cuda_lib, shift):
    """A single row whose label lies below the other logits, within the tile's range (50 nats) and beyond it."""
    torch = _torch()
    N, d, V = 300, 64, 80101
    rng, H, W, y = make(N, d, V, seed=5)
    row = int(np.flatnonzero(y >= 0)[10])
    W[:, 0] = 0.0
    H[:, 0] = 0.0
    W[y[row], 0] = -1.0
    H[row, 0] = shift                       # z_y of this row falls by that much; no other row sees it
    Ht, Wt = heads(H, W)
    inp = policy_inputs(rng, H, W, y, 1.0)
    kw = dict(clip_low=0.2, clip_high=0.28, kl="k3", kl_coef=0.1)
    check_policy(call_policy(cuda_lib, Ht, Wt, dev(y), inp, sync_check=True, **kw), H, W, y, inp, **kw)
    cu = bounds(rng, N, 3)
    check_preference(call_preference(cuda_lib, Ht, Wt, y, cu, None, average=True, sync_check=True), H, W, y, cu, None, average=True)


def test_exp_tiles_of_confident_rows(cuda_lib):
    """A label with nearly all of the probability: logp near 0 and the gradient of 1 - p keep their relative precision."""
    N, d, V = 300, 64, 80101
    rng, H, W, _ = make(N, d, V, seed=6, peak=0.0)
    y = np.full(N, 7)
    W[:, 0] = 0.0
    W[7] = 0.0
    W[7, 0] = 1.0
    H[:, 0] = np.round(4 * (20.0 + 40.0 * rng.random(N))) / 4    # z_y; the others are below 20: 1 - p from 1e-2 to 1e-18
    Ht, Wt = heads(H, W)
    inp = dict(advantages=f32(np.ones(N)), old_logp=None, ref_logp=None, weights=None)
    _, logp, _, dH, _ = call_policy(cuda_lib, Ht, Wt, dev(y), inp)
    z = H @ W.T
    others = np.exp(z - z[:, 7:8])
    others[:, 7] = 0.0
    rest = others.sum(axis=1)
    assert rest.min() < 1e-10
    np.testing.assert_allclose(np64(logp), -np.log1p(rest), rtol=2.0 ** -15)
    G = others / (1 + rest)[:, None]
    G[:, 7] = -rest / (1 + rest)
    want, bulk = G @ W / N, np.abs(G) @ np.abs(W) / N
    close(dH, want, (2 * U + U * U + 2.0 ** -10) * bulk + U * np.abs(want), "dH")


# --------------------------------------------------------------------------- layer norm
def norm_inputs(N, d, seed=0, offset=0.0, f32_x=False):
    torch = _torch()
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((N, d)) * (0.5 + 4 * rng.random((N, 1))) + offset
    x = dev(x).to(torch.float32 if f32_x else torch.bfloat16)
    dH = dev(rng.standard_normal((N, d))).to(torch.bfloat16)
    return rng, x, dH


def check_norm(lce, x, w, b, dH, eps=1e-5):
    torch = _torch()
    N, d = x.shape
    X, G = np64(x), np64(dH)
    w64, b64 = (None if t is None else np64(t) for t in (w, b))
    H, mean, rstd = lce.lce_layernorm_forward(x, w, b, eps)
    ref = oracle.layernorm_f64(X, w64, b64, float(np.float32(eps)))
    g = (d / 32 + 16) * EPS
    em = g * np.abs(X).mean(axis=1) + 2.0 ** -149
    r = ref["rstd"]
    rel = 2 * g + (em * r) ** 2 + 2.0 ** -21
    close(mean, ref["mean"], em + EPS * np.abs(ref["mean"]), "mean")
    close(rstd, r, r * rel, "rstd")
    xh = oracle.layernorm_f64(X, None, None, float(np.float32(eps)))["H"]
    ex = (r * em)[:, None] + np.abs(xh) * rel[:, None]
    aw = 1.0 if w is None else np.abs(w64)
    tol = aw * ex + 2.0 ** -21 * (np.abs(xh) * aw + (0 if b is None else np.abs(b64)))
    close(H, ref["H"], tol * (1 + U) + U * np.abs(ref["H"]) + 1e-38, "H")
    back = oracle.layernorm_backward_f64(X, w64, G, float(np.float32(eps)))
    ag = np.abs(G) * aw
    c = np.abs((G * (1.0 if w is None else w64) * xh).sum(axis=1, keepdims=True)) / d
    tol_dx = (3 * g + 2.0 ** -20 + rel[:, None]) * back["dx_bulk"] + r[:, None] * (
        ex * c + np.abs(xh) * (ag * ex).sum(axis=1, keepdims=True) / d)
    out = U * np.abs(back["dx"]) if x.dtype == torch.bfloat16 else 0.0
    tol_dw = (np.abs(G) * ex).sum(axis=0) + (N * EPS + 2.0 ** -21) * back["dw_bulk"] + 1e-38
    tol_db = (N * EPS + 2.0 ** -21) * back["db_bulk"] + 1e-38
    dx, dw, db = lce.lce_layernorm_backward(x, w, mean, rstd, dH)
    assert dx.dtype == x.dtype and (dw is None) == (w is None)
    close(dx, back["dx"], tol_dx * (1 + U) + out + 1e-38, "dx")
    if dw is not None:
        close(dw, back["dw"], tol_dw, "dw")
    close(db, back["db"], tol_db, "db")
    # each of them alone, and the same again
    for kw, at in ((dict(bias=False, need_dw=False), 0), (dict(bias=False, need_dx=False), 1), (dict(need_dx=False, need_dw=False), 2)):
        if at == 1 and w is None:
            continue
        got = lce.lce_layernorm_backward(x, w, mean, rstd, dH, **kw)
        for k in range(3):
            assert torch.equal(got[k], (dx, dw, db)[k]) if k == at else got[k] is None


NORM_CASES = [(1, 8), (2, 24), (3, 256), (1, 2048), (5, 264), (33, 520), (7, 1032), (64, 2048), (17, 2056), (300, 4096),
              (9, 4104), (4, 8192), (5, 8200), (3, 16384), (2, 32768), (1000, 264), (2049, 72), (700, 1024)]


@pytest.mark.parametrize("N,d", NORM_CASES)
@pytest.mark.parametrize("f32_x", [False, True])
def test_layernorm(cuda_lib, N, d, f32_x):
    torch = _torch()
    rng, x, dH = norm_inputs(N, d, seed=N + d, f32_x=f32_x)
    w, b = dev(f32(1 + 0.3 * rng.standard_normal(d))), dev(f32(rng.standard_normal(d)))
    check_norm(cuda_lib, x, w, b, dH)
    check_norm(cuda_lib, x, w.bfloat16(), b.bfloat16(), dH)
    check_norm(cuda_lib, x, w, None, dH)
    check_norm(cuda_lib, x, None, None, dH, eps=1e-3)


@pytest.mark.parametrize("d", [64, 1000, 4096])
def test_layernorm_far_means_and_flat_rows(cuda_lib, d):
    """Rows whose mean is far larger than their deviation, rows of one value, tiny and huge rows, eps = 0."""
    torch = _torch()
    rng, x, dH = norm_inputs(20, d, offset=1000.0, f32_x=True)
    w, b = dev(f32(1 + 0.3 * rng.standard_normal(d))), dev(f32(rng.standard_normal(d)))
    check_norm(cuda_lib, x, w, b, dH)
    _, x, dH = norm_inputs(20, d, f32_x=True)
    check_norm(cuda_lib, x * 1e-12, w, b, dH, eps=0.0)
    check_norm(cuda_lib, x * 1e12, w, b, dH)
    flat = torch.full((6, d), 0.75, device="cuda")
    H, mean, rstd = cuda_lib.lce_layernorm_forward(flat, w, b)
    assert torch.equal(H, b.bfloat16().expand(6, d)) and (mean == 0.75).all()
    np.testing.assert_allclose(np64(rstd), 1e-5 ** -0.5, rtol=1e-6)


def test_layernorm_rows_of_nan_leave_the_others_alone(cuda_lib):
    torch = _torch()
    rng, x, dH = norm_inputs(50, 264)
    w = dev(f32(1 + 0.3 * rng.standard_normal(264)))
    H, mean, rstd = cuda_lib.lce_layernorm_forward(x, w)
    bad = x.clone()
    bad[7] = float("nan")
    bad[20, 3] = float("inf")
    H2, mean2, rstd2 = cuda_lib.lce_layernorm_forward(bad, w)
    keep = torch.ones(50, dtype=torch.bool, device="cuda")
    keep[[7, 20]] = False
    assert torch.equal(H2[keep], H[keep]) and H2[7].isnan().all() and H2[20].isnan().any()
    dx = cuda_lib.lce_layernorm_backward(x, w, mean, rstd, dH)[0]
    dx2 = cuda_lib.lce_layernorm_backward(bad, w, mean2, rstd2, dH)[0]
    assert torch.equal(dx2[keep], dx[keep])


def test_layernorm_no_rows(cuda_lib):
    torch = _torch()
    x = torch.zeros(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    H, mean, rstd = cuda_lib.lce_layernorm_forward(x, w, w)
    dx, dw, db = cuda_lib.lce_layernorm_backward(x, w, mean, rstd, H)
    assert H.shape == dx.shape == (0, 64) and not dw.any() and not db.any()


def test_layernorm_past_32_bits(cuda_lib):
    """Offsets past 2^31 elements: the last rows are those of a call of their own; dw of rows that are all alike."""
    torch = _torch()
    N, d = 70000, 32768
    x = torch.zeros(N, d, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(100, d, device="cuda").bfloat16()
    x[-100:] = tail
    dH = x.clone()
    H, mean, rstd = cuda_lib.lce_layernorm_forward(x)
    Ht, mt, rt = cuda_lib.lce_layernorm_forward(tail)
    assert torch.equal(H[-100:], Ht) and torch.equal(mean[-100:], mt) and torch.equal(rstd[-100:], rt) and not H[:-100].any()
    dx, _, db = cuda_lib.lce_layernorm_backward(x, None, mean, rstd, dH)
    dxt, _, dbt = cuda_lib.lce_layernorm_backward(tail, None, mt, rt, tail)
    assert torch.equal(dx[-100:], dxt) and not dx[:-100].any()
    assert ((db - dbt).abs() <= 200 * EPS * tail.float().abs().sum(0)).all()


def test_layernorm_short_rows_and_long_batches(cuda_lib):
    """Many rows of few elements, whose gradients many blocks share, and the one-pass backward past 2^31 elements."""
    torch = _torch()
    for N in (2048, 2049, 60001):
        rng, x, dH = norm_inputs(N, 8, seed=N)
        check_norm(cuda_lib, x, dev(f32(1 + 0.1 * rng.standard_normal(8))), dev(f32(rng.standard_normal(8))), dH)
    N, d = 270000, 8192
    x = torch.zeros(N, d, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(100, d, device="cuda").bfloat16()
    x[-100:] = tail
    w = torch.ones(d, device="cuda")
    H, mean, rstd = cuda_lib.lce_layernorm_forward(x, w)
    Ht, mt, rt = cuda_lib.lce_layernorm_forward(tail, w)
    assert torch.equal(H[-100:], Ht) and torch.equal(mean[-100:], mt) and torch.equal(rstd[-100:], rt) and not H[:-100].any()
    dx, dw, db = cuda_lib.lce_layernorm_backward(x, w, mean, rstd, x)
    dxt, dwt, dbt = cuda_lib.lce_layernorm_backward(tail, w, mt, rt, tail)
    assert torch.equal(dx[-100:], dxt) and not dx[:-100].any()
    assert ((db - dbt).abs() <= 200 * EPS * tail.float().abs().sum(0)).all()
    xh = (tail.float() - mt[:, None]) * rt[:, None]
    assert ((dw - dwt).abs() <= 200 * EPS * (xh * tail.float()).abs().sum(0)).all()


# --------------------------------------------------------------------------- together
def step_inputs(N, d, V, seed=3):
    torch = _torch()
    rng, H, W, y = make(N, d, V, seed=seed)
    x = dev(H, torch.bfloat16)
    w = dev(f32(1 + 0.1 * rng.standard_normal(d)))
    b = dev(f32(0.1 * rng.standard_normal(d)))
    _, Wt = heads(H, W)
    return rng, x, w, b, Wt, y


def test_norm_head_and_losses_together(cuda_lib):
    """A training step through the modules: layer norm, head, policy and preference loss; its gradients against
    those of the oracle for the hidden states the norm gave."""
    torch = _torch()
    from chunked_lm_head_linear_gb300.autograd import FusedLayerNorm, FusedLinearPolicyLoss, FusedLinearPreferenceLoss
    N, d, V = 160, 64, 1200
    rng, x, w, b, Wt, y = step_inputs(N, d, V)
    x, w, b, Wt = (t.requires_grad_(True) for t in (x, w, b, Wt))
    cu = bounds(rng, N, 3, 0, 5)
    norm = FusedLayerNorm()
    H = norm(x, w, b)
    H64, W64 = np64(H), np64(Wt)
    logp, told, _ = head(H64, W64, y, 1.0)
    inp = dict(advantages=f32(rng.standard_normal(N)), old_logp=f32(np.where(told, logp - 0.05, 0.0)), ref_logp=f32(logp - 0.3),
               weights=None)
    args = [None if inp[k] is None else dev(inp[k]) for k in ("advantages", "old_logp", "ref_logp", "weights")]
    loss, got_logp = FusedLinearPolicyLoss(kl="k3", kl_coef=0.2)(H, Wt, dev(y), *args)
    pref, seq = FusedLinearPreferenceLoss(beta=0.2)(H, Wt, dev(y), dev(cu))
    assert not got_logp.requires_grad and not seq.requires_grad
    dH, dW = torch.autograd.grad(2.0 * loss + 0.5 * pref, [H, Wt], retain_graph=False)
    one = oracle.policy_f64(H64, W64, y, *[None if inp[k] is None else inp[k].astype(np.float64) for k in
                            ("advantages", "old_logp", "ref_logp", "weights")], kl="k3", kl_coef=0.2, grad_loss=2.0)
    two = oracle.preference_f64(H64, W64, y, cu, beta=0.2, grad_loss=0.5)
    ref = {k: one[k] + two[k] for k in ("dH", "dW", "dH_bulk", "dW_bulk")}
    # two gradients of one rounding each, and the rounding of their sum
    extra = {k + "_bulk": 2 * U * (np.abs(one[k]) + np.abs(two[k])) + 2.0 ** -9 * ref[k + "_bulk"] for k in ("dH", "dW")}
    check_gradients(dH, dW, ref, extra)
    # the whole step down to the norm's input and parameters
    loss, _ = FusedLinearPolicyLoss(kl="k3", kl_coef=0.2)(norm(x, w, b), Wt, dev(y), *args)
    dx, dw, db, _ = torch.autograd.grad(loss, [x, w, b, Wt])
    back = oracle.layernorm_backward_f64(np64(x), np64(w), one["dH"] / 2.0)
    for got, k in ((dx, "dx"), (dw, "dw"), (db, "db")):
        assert np.linalg.norm(np64(got) - back[k]) <= 1e-2 * np.linalg.norm(back[k]), k   # dH's 5e-3 and the roundings of dH and dx


def _step(lce, x, w, b, Wt, yt, cu, inp, ws=None, stream=None):
    H, mean, rstd = lce.lce_layernorm_forward(x, w, b, stream=stream)
    out = [H, mean, rstd]
    out += lce.lce_policy_fwd_bwd(H, Wt, yt, inp[0], inp[1], inp[2], kl="k3", kl_coef=0.1, workspace=ws, stream=stream)
    out += lce.lce_policy_forward(H, Wt, yt, inp[0], inp[1], workspace=ws, stream=stream)
    out += lce.lce_preference_fwd_bwd(H, Wt, yt, cu, dW_dtype=_torch().bfloat16, workspace=ws, stream=stream)
    out += lce.lce_layernorm_backward(x, w, mean, rstd, out[6], stream=stream)
    return out


@pytest.mark.parametrize("N,chunk", [(8, 0), (300, 0), (300, 128)])
def test_streams_graphs_and_a_shared_workspace(cuda_lib, N, chunk):
    """The calls on a side stream, two at once, captured once and replayed on other inputs, all with one workspace."""
    torch = _torch()
    d, V = 64, 3001
    rng, x, w, b, Wt, y = step_inputs(N, d, V)
    yt, cu = dev(y), dev(bounds(rng, N, 2))
    logp = dev(f32(-8.0 + rng.standard_normal(N)))
    inp = (dev(f32(rng.standard_normal(N))), logp, logp + 0.1)
    need = max(cuda_lib.lce_policy_workspace_size(N, d, V), cuda_lib.lce_preference_workspace_size(N, d, V, 2, True, 1))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    other = x.flip(0).contiguous()
    want = [_step(cuda_lib, t, w, b, Wt, yt, cu, inp, ws) for t in (x, other)]
    fresh = _step(cuda_lib, x, w, b, Wt, yt, cu, inp)
    torch.cuda.synchronize()
    for a, c in zip(want[0], fresh):
        assert torch.equal(a, c)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = _step(cuda_lib, x, w, b, Wt, yt, cu, inp, ws)
    side.synchronize()
    for a, c in zip(want[0], got):
        assert torch.equal(a, c)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        got = [_step(cuda_lib, t, w, b, Wt, yt, cu, inp, stream=s) for t, s in zip((x, other), streams)]
        torch.cuda.synchronize()
        for k in range(2):
            for a, c in zip(want[k], got[k]):
                assert torch.equal(a, c)
    buf = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _step(cuda_lib, buf, w, b, Wt, yt, cu, inp, ws)
    for k in (1, 0, 1):
        buf.copy_((x, other)[k])
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(want[k], out):
            assert torch.equal(a, c)


def test_modules_captured_and_replayed(cuda_lib):
    """A whole step through the modules, captured once and replayed on other hidden states."""
    torch = _torch()
    from chunked_lm_head_linear_gb300.autograd import FusedLayerNorm, FusedLinearPolicyLoss, FusedLinearPreferenceLoss
    N, d, V = 200, 64, 700
    rng, x0, w, b, Wt, y = step_inputs(N, d, V)
    yt, cu, A = dev(y), dev(bounds(rng, N, 2)), dev(f32(rng.standard_normal(N)))
    x, w, b, Wt = (t.clone().requires_grad_(True) for t in (x0, w, b, Wt))

    def step():
        H = FusedLayerNorm()(x, w, b)
        loss, _ = FusedLinearPolicyLoss()(H, Wt, yt, A)
        pref, _ = FusedLinearPreferenceLoss()(H, Wt, yt, cu)
        return [loss, pref, *torch.autograd.grad(loss + pref, [x, w, b, Wt])]

    want = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for k in range(2):
            with torch.no_grad():
                x.copy_(x0 if k == 0 else -x0)
            want.append([o.detach().clone() for o in step()])
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in (0, 1, 0):
        with torch.no_grad():
            x.copy_(x0 if k == 0 else -x0)
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(out, want[k]):
            assert torch.equal(a, c)


def test_what_does_not_fit_is_refused(cuda_lib):
    torch = _torch()
    _, H, W, y = make(20, 64, 300)
    Ht, Wt, yt = *heads(H, W), dev(y)
    f, cu = torch.zeros(20, device="cuda"), torch.tensor([0, 5, 20], device="cuda")
    L = cuda_lib
    for call in (lambda: L.lce_policy_forward(Ht.float(), Wt, yt, f), lambda: L.lce_policy_forward(Ht, Wt, yt, f[:5]),
                 lambda: L.lce_policy_forward(Ht, Wt, yt, f.double()), lambda: L.lce_policy_forward(Ht, Wt, yt, None),
                 lambda: L.lce_policy_forward(Ht, Wt, yt, f, f.cpu()), lambda: L.lce_policy_fwd_bwd(Ht, Wt, yt, f, kl="k3"),
                 lambda: L.lce_policy_fwd_bwd(Ht, Wt, yt, f, kl="kl"), lambda: L.lce_policy_fwd_bwd(Ht, Wt, yt, f, weights=f[:3]),
                 lambda: L.lce_policy_fwd_bwd(Ht, Wt, yt, f, need_dH=False, need_dW=False),
                 lambda: L.lce_policy_fwd_bwd(Ht, Wt, yt, f, accumulate_dW=True),
                 lambda: L.lce_preference_forward(Ht, Wt, yt, cu[:2]), lambda: L.lce_preference_forward(Ht, Wt, yt, cu.float()),
                 lambda: L.lce_preference_forward(Ht, Wt, yt, cu.cpu()), lambda: L.lce_preference_forward(Ht, Wt, yt, cu, f),
                 lambda: L.lce_preference_forward(Ht, Wt, yt, cu, kind="dpo"),
                 lambda: L.lce_preference_forward(Ht, Wt, yt, cu, kind="ipo", margin=1.0),
                 lambda: L.lce_preference_fwd_bwd(Ht, Wt, yt, cu, kind="hinge", label_smoothing=0.1),
                 lambda: L.lce_layernorm_forward(Ht.half()), lambda: L.lce_layernorm_forward(Ht.t()),
                 lambda: L.lce_layernorm_forward(Ht, f), lambda: L.lce_layernorm_forward(Ht, torch.ones(64, device="cuda"),
                                                                                        torch.ones(64, device="cuda").bfloat16()),
                 lambda: L.lce_layernorm_backward(Ht, None, f, f, Ht.float()), lambda: L.lce_layernorm_backward(Ht, None, f, None, Ht),
                 lambda: L.lce_layernorm_backward(Ht, None, f, f, Ht, bias=False, need_dx=False)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: L.lce_policy_forward(Ht, Wt, yt, f, clip_low=-1.0), lambda: L.lce_policy_forward(Ht, Wt, yt, f, dual_clip=0.5),
                 lambda: L.lce_policy_forward(Ht, Wt, yt, f, temperature=0.0), lambda: L.lce_preference_forward(Ht, Wt, yt, cu, beta=0.0),
                 lambda: L.lce_layernorm_forward(Ht, eps=-1.0), lambda: L.lce_layernorm_forward(torch.zeros(4, 12, device="cuda"))):
        with pytest.raises(L.LCEError) as err:
            call()
        assert err.value.code == L.LCE_ERR_INVALID_ARG
    small = torch.empty(1000, dtype=torch.uint8, device="cuda")
    for call in (lambda: L.lce_policy_forward(Ht, Wt, yt, f, workspace=small),
                 lambda: L.lce_preference_fwd_bwd(Ht, Wt, yt, cu, workspace=small),
                 lambda: L.lce_layernorm_backward(Ht, None, f, f, Ht, workspace=small[:100])):
        with pytest.raises(L.LCEError) as err:
            call()
        assert err.value.code == L.LCE_ERR_WORKSPACE
    for a, c in zip(L.lce_policy_fwd_bwd(Ht, Wt, yt, f + 1, chunk_tokens="auto"), L.lce_policy_fwd_bwd(Ht, Wt, yt, f + 1)):
        assert torch.equal(a, c)


# --------------------------------------------------------------------------- the bounds-checking build
def _child():
    """Every kind of call on the bounds-checking build (a process loads one library)."""
    from chunked_lm_head_linear_gb300 import build, lce
    lce.load(build.build(checks=True))
    torch = _torch()
    for N, d, V, chunk in [(1, 64, 37, 0), (3, 72, 2, 0), (96, 64, 4099, 0), (97, 8, 257, 0), (129, 136, 70001, 64),
                           (513, 256, 1000, 200), (400, 64, 30001, 0), (100, 64, 250007, 0), (300, 64, 100003, 250)]:
        rng, H, W, y = make(N, d, V, seed=N)
        Ht, Wt = heads(H, W)
        inp = policy_inputs(rng, H, W, y, 1.0, "k3")
        kw = dict(clip_low=0.2, clip_high=0.28, kl="k3", kl_coef=0.1)
        for grad in (True, False):
            out = call_policy(lce, Ht, Wt, dev(y), inp, grad=grad, chunk_tokens=chunk, sync_check=True, **kw)
            check_policy(out, H, W, y, inp, chunk=chunk, **kw)
            cu = bounds(rng, N, 2)
            out = call_preference(lce, Ht, Wt, y, cu, None, grad=grad, chunk_tokens=chunk, sync_check=True)
            check_preference(out, H, W, y, cu, None, chunk=chunk)
        check_norm(lce, Ht, torch.ones(d, device="cuda"), None, Ht)
    print("checked build: ok")


def test_bounds_checking_build(cuda_lib):
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([os.path.dirname(here), here]))
    r = subprocess.run([sys.executable, "-c", "import test_losses_gpu as t; t._child()"], env=env, cwd=here,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "checked build: ok" in r.stdout, (r.stdout + r.stderr)[-3000:]
