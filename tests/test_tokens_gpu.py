"""The head's token operators on the GPU against the fp64 oracle.

Inputs lie on a grid (H on 1/16 and W on 1/64, at most 7 bits and a sign), so
every logit is a whole multiple of 2^-10 below 2^24 of them and exact in fp32
in any order of its sum: the alternatives, ties included, are the oracle's.

Tolerances, with z' = z / T, D the largest |z'| spread, eps = 2^-24 (fp32) and
u = 2^-8 (bf16):
  lse, logp    each exponential errs by 2^-22 (ex2.approx) and by the rounding
               of its argument, 3 eps |z' - m| (weighted by p it averages below
               3 eps (entropy + 1) <= 3 eps 13); a sum in fp32 over 32 terms, 4
               groups and the merges of up to 1200 half tiles adds at most
               (32 + 4 + 40 + 12) eps; the final sum rounds eps |lse|, z / T
               eps |z'|: together below 2^-16 + 2^-21 (|lse| + |z'|)
  entropy      log S - T/S: the same relative errors on S and on T, T/S up to
               ln V <= 12: 13 times the bound above
  gradients    each entry of G is rounded to bf16 once (u), its factors err by
               less than 2^-10 relative (lse and entropy as above, up to 13
               nats): every element of distillation's dW lies within (u + 2^-10)
               bulk, bulk the sum of the absolute terms it is made of; dW of
               log-probabilities within (2 u + u^2 + 2^-10) bulk, its other
               operand bf16(scale H) being rounded as well; dH within (u + 2^-10)
               bulk plus its own rounding u |dH|; whole tensors within 5e-3
               (rounding errors average: u / sqrt(3) each). Where log p + entropy
               cancels, its absolute error, 14 times that of lse (2^-12), stays:
               2^-12 times the sums over p |e| on top.
"""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


def _torch():
    import torch
    return torch


def grid(x, steps):
    return np.clip(np.round(x * steps), -127, 127) / steps


def dev(x, dtype=None):
    torch = _torch()
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def make(N, d, V, seed=0, scale=2.0, peak=8.0):
    """H, W (fp64, on the grid), labels with some ignored; rows lean towards their label."""
    rng = np.random.default_rng(seed)
    sigma = scale / np.sqrt(d)
    W = grid(rng.standard_normal((V, d)) * min(1.0, sigma), 64)
    y = rng.integers(0, V, N)
    H = rng.standard_normal((N, d)) + W[y] * (peak * rng.random((N, 1)) / (sigma * sigma * d))
    H = grid(H, 16)
    y[rng.random(N) < 0.15] = oracle.IGNORE_INDEX
    return rng, H, W, y.astype(np.int64)


def heads(H, W):
    torch = _torch()
    return dev(H, torch.bfloat16), dev(W, torch.bfloat16)


def np64(t):
    return t.detach().double().cpu().numpy()


def close(got, ref, tol, what):
    err = np.abs(np64(got) - ref)
    assert np.all(err <= tol), f"{what}: off by {np.nanmax(err):.3e}, {np.nanmax(err / tol):.2f} of the bound"


def tol_lse(H, W, lse, T):
    zmax = np.abs(H @ W.T).max(axis=1) / T
    return 2.0 ** -16 + 2.0 ** -21 * (np.abs(lse) + zmax)


def check_scores(out, H, W, y, T, K):
    logp, lse, ent, tl, ti = out
    ref = oracle.logprobs_f64(H, W, y, temperature=T, top_k=K)
    tol = tol_lse(H, W, ref["lse"], T)
    close(lse, ref["lse"], tol, "lse")
    close(logp, ref["logp"], 2 * tol, "logp")
    if ent is not None:
        close(ent, ref["entropy"], 13 * tol, "entropy")
    if K:
        assert (ti.cpu().numpy() == ref["top_idx"]).all(), "alternatives"
        close(tl, ref["top_logp"], 2 * tol[:, None], "top_logp")
    return ref


def check_grads(dH, dW, ref, scaled=False):
    """scaled: dW's second operand is rounded too (log-probabilities)."""
    for got, name in ((dH, "dH"), (dW, "dW")):
        if got is None:
            continue
        u = 2 * U + U * U if scaled and name == "dW" else U
        out = U * np.abs(ref[name]) if got.dtype == _torch().bfloat16 else 0.0
        slack = 2.0 ** -12 * ref[name + "_slack"] if scaled and name + "_slack" in ref else 0.0
        close(got, ref[name], (u + 2.0 ** -10) * ref[name + "_bulk"] + slack + out + 1e-30, name)
        norm = np.linalg.norm(ref[name])
        assert np.linalg.norm(np64(got) - ref[name]) <= 5e-3 * norm, name


# N, d, V, K, T, chunk
SCORE_CASES = [
    (1, 8, 1, 1, 1.0, 0),            # one token, one word
    (1, 64, 37, 5, 1.0, 0),          # one decoded token
    (3, 72, 2, 2, 0.7, 0),           # K tail, two words, both returned
    (5, 64, 128, 128, 2.0, 0),       # every word of one half tile returned
    (16, 128, 129, 33, 1.0, 0),      # one column in the second half tile
    (33, 64, 5003, 64, 0.5, 0),
    (64, 256, 4096, 8, 1.0, 0),
    (65, 256, 4096, 1, 1.0, 0),
    (100, 136, 12345, 40, 1.3, 0),
    (129, 136, 4099, 20, 1.0, 64),   # chunks smaller than a tile
    (257, 264, 1000, 0, 1.0, 0),     # no alternatives
    (300, 264, 5003, 128, 1.0, 128),
    (513, 256, 1000, 7, 1.3, 200),   # chunks that are not a multiple of the tile
    (2, 64, 151655, 20, 1.0, 0),     # the unpadded vocabulary
    (130, 64, 70001, 9, 1.0, 0),
    (37, 64, 333, 5, 1e-6, 0),       # the coldest: one token, or several equal ones, have all of it
    (130, 64, 333, 5, 1e6, 0),       # the hottest: all but uniform
]


@pytest.mark.parametrize("N,d,V,K,T,chunk", SCORE_CASES)
def test_logprobs(cuda_lib, N, d, V, K, T, chunk):
    _, H, W, y = make(N, d, V, seed=N + V)
    Ht, Wt = heads(H, W)
    out = cuda_lib.lce_logprobs(Ht, Wt, dev(y), top_k=K, temperature=T, chunk_tokens=chunk, sync_check=True)
    check_scores(out, H, W, y, T, K)
    if K:   # the statistics do not depend on how many alternatives are asked for
        logp, lse, ent, tl, ti = cuda_lib.lce_logprobs(Ht, Wt, dev(y), temperature=T, chunk_tokens=chunk, entropy=False)
        assert ent is None and tl is None and ti is None
        check_scores((logp, lse, None, None, None), H, W, y, T, 0)


@pytest.mark.parametrize("N", [1, 40, 300])
def test_logprobs_ties_go_to_the_lowest_index(cuda_lib, N):
    """All logits equal, and logits of three values only: many ties inside and across tiles."""
    torch = _torch()
    V, d, K = 1500, 64, 37
    y = torch.zeros(N, dtype=torch.int64, device="cuda")
    out = cuda_lib.lce_logprobs(torch.ones(N, d, dtype=torch.bfloat16, device="cuda"),
                                torch.zeros(V, d, dtype=torch.bfloat16, device="cuda"), y, top_k=K)
    assert (out[4] == torch.arange(K, device="cuda")).all()
    assert (out[2] - float(np.log(V))).abs().max() < 13 * 2.0 ** -15
    W = np.zeros((V, d))
    W[:, 0] = np.random.default_rng(1).integers(-1, 2, V)
    H = np.zeros((N, d))
    H[:, 0] = np.where(np.arange(N) % 2 == 0, 1.0, -1.0)   # the order turns round in every other row
    Ht, Wt = heads(H, W)
    check_scores(cuda_lib.lce_logprobs(Ht, Wt, y, top_k=K), H, W, y.cpu().numpy(), 1.0, K)


@pytest.mark.parametrize("N", [2, 300])
def test_logprobs_far_logits(cuda_lib, N):
    """Spreads of hundreds of nats: probabilities underflow, entropy goes to zero, nothing overflows."""
    _, H, W, y = make(N, 64, 3000, scale=8.0, peak=0.0)
    H = H * 8
    Ht, Wt = heads(H, W)
    assert np.abs(H @ W.T).max() > 150
    check_scores(cuda_lib.lce_logprobs(Ht, Wt, dev(y), top_k=12), H, W, y, 1.0, 12)


@pytest.mark.parametrize("N", [3, 200])
def test_logprobs_near_zero_keep_their_relative_precision(cuda_lib, N):
    """A confident row: logp = -log1p(s) with s down to e^-30. Each term of s errs by 2^-22 and by its
    argument's rounding, 2 eps |z' - m| < 2^-17; the sum and log1p by far less: below 2^-16 relative."""
    V, d, label = 5000, 64, 1234
    W = np.zeros((V, d))
    W[:, 0] = -1.0
    W[label, 0] = 0.0
    W[:, 1] = np.random.default_rng(5).integers(-8, 9, V) / 64
    H = np.zeros((N, d))
    H[:, 0] = 20 + np.arange(N) % 11      # the label's lead over the others, in nats
    H[:, 1] = 1.0
    y = np.full(N, label)
    Ht, Wt = heads(H, W)
    logp, _, ent, tl, ti = cuda_lib.lce_logprobs(Ht, Wt, dev(y), top_k=1)
    ref = oracle.logprobs_f64(H, W, y, top_k=1)
    z = H @ W.T
    exact = -np.log1p(np.exp(np.delete(z, label, axis=1) - z[:, [label]]).sum(axis=1))
    assert exact.max() < 0 and exact.min() > -1e-4 and (ti.cpu().numpy() == label).all()
    close(logp, exact, 2.0 ** -16 * np.abs(exact), "logp")
    close(tl[:, 0], exact, 2.0 ** -16 * np.abs(exact), "top_logp")
    # entropy = log1p(s) - t / (1 + s), two positive parts
    close(ent, ref["entropy"], 2.0 ** -15 * np.abs(ref["entropy"]) + 1e-12, "entropy")


@pytest.mark.parametrize("N", [4, 300])
def test_logprobs_rows_with_nan_and_inf_leave_the_others_alone(cuda_lib, N):
    torch = _torch()
    _, H, W, y = make(N, 64, 2000)
    Ht, Wt = heads(H, W)
    clean = cuda_lib.lce_logprobs(Ht, Wt, dev(y), top_k=16)
    Ht[1, 3] = float("nan")
    Ht[2, 5] = float("inf")
    logp, lse, ent, tl, ti = cuda_lib.lce_logprobs(Ht, Wt, dev(y), top_k=16)
    rest = torch.tensor([i for i in range(N) if i not in (1, 2)], device="cuda")
    for a, b in zip((logp, lse, ent, tl, ti), clean):
        assert torch.equal(a[rest], b[rest])
    assert torch.isnan(lse[1]) and torch.isnan(ent[1])
    assert ((ti >= 0) & (ti < 2000)).all()


def test_logprobs_label_out_of_range(cuda_lib):
    torch = _torch()
    _, H, W, y = make(50, 64, 300)
    Ht, Wt = heads(H, W)
    yt = dev(y)
    yt[7], yt[9] = 300, -5
    with pytest.raises(cuda_lib.LCEError) as err:
        cuda_lib.lce_logprobs(Ht, Wt, yt, sync_check=True)
    assert err.value.code == cuda_lib.LCE_ERR_LABEL_RANGE
    out = cuda_lib.lce_logprobs(Ht, Wt, yt, top_k=4)
    y[7] = y[9] = oracle.IGNORE_INDEX
    check_scores(out, H, W, y, 1.0, 4)
    assert torch.equal(out[0][7], torch.zeros((), device="cuda"))


def test_ignore_index_inside_the_vocabulary(cuda_lib):
    """A padding id that is a word: equality with it comes first, in labels and in teacher entries."""
    rng, H, W, y = make(120, 64, 300)
    y = rng.integers(0, 8, 120)
    Ht, Wt = heads(H, W)
    out = cuda_lib.lce_logprobs(Ht, Wt, dev(y), top_k=3, ignore_index=5, sync_check=True)
    ref = oracle.logprobs_f64(H, W, y, top_k=3, ignore_index=5)
    close(out[0], ref["logp"], 2 * tol_lse(H, W, ref["lse"], 1.0), "logp")
    assert not out[0][dev(y == 5)].any() and (y == 5).any()
    g = rng.standard_normal(120).astype(np.float32)
    dH, dW = cuda_lib.lce_logprobs_backward(Ht, Wt, dev(y), *out[:3], dev(g), dev(g), ignore_index=5)
    check_grads(dH, dW, oracle.logprobs_backward_f64(H, W, y, g, g, ignore_index=5), scaled=True)
    idx = rng.integers(0, 8, (120, 4))
    t = rng.standard_normal((120, 4)).astype(np.float32)
    _, _, dH, dW = cuda_lib.lce_distill_fwd_bwd(Ht, Wt, dev(idx), dev(t), ignore_index=5, sync_check=True)
    check_grads(dH, dW, oracle.distill_f64(H, W, idx, t, ignore_index=5))


@pytest.mark.parametrize("N", [40, 300])
def test_a_wait_that_runs_out_is_reported(cuda_lib, N):
    """No operand is loaded, so the bounded waits of the logits kernels run out (about 2 s): the call
    returns LCE_ERR_TIMEOUT, and the next one works."""
    _, H, W, y = make(N, 64, 1000)
    Ht, Wt = heads(H, W)
    with pytest.raises(cuda_lib.LCEError) as err:
        cuda_lib.lce_logprobs(Ht, Wt, dev(y), top_k=4, sync_check=True, reserved=cuda_lib.LCE_TEST_FORCE_TIMEOUT)
    assert err.value.code == cuda_lib.LCE_ERR_TIMEOUT
    check_scores(cuda_lib.lce_logprobs(Ht, Wt, dev(y), top_k=4, sync_check=True), H, W, y, 1.0, 4)


def test_logprobs_no_tokens(cuda_lib):
    torch = _torch()
    H, W = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(9, 64, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(0, dtype=torch.int64, device="cuda")
    logp, lse, ent, tl, ti = cuda_lib.lce_logprobs(H, W, y, top_k=3)
    assert logp.shape == lse.shape == ent.shape == (0,) and tl.shape == ti.shape == (0, 3)
    dH, dW = cuda_lib.lce_logprobs_backward(H, W, y, logp, lse, ent, logp, ent)
    assert dH.shape == (0, 64) and not dW.any()
    idx = torch.zeros(0, 4, dtype=torch.int64, device="cuda")
    loss, row, dH, dW = cuda_lib.lce_distill_fwd_bwd(H, W, idx, idx.float())
    assert loss.item() == 0 and row.shape == (0,) and not dW.any()


def test_logprobs_logits_buffer_past_32_bits(cuda_lib):
    """A chunk whose logits take 16384 x 151808 entries (more than 2^31) equals small chunks bit for bit."""
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(3)
    H = (torch.randn(16384, 64, generator=g, device="cuda") * 16).round().clamp(-127, 127).div(16).bfloat16()
    W = (torch.randn(151655, 64, generator=g, device="cuda") * 16).round().clamp(-127, 127).div(64).bfloat16()
    y = torch.randint(0, 151655, (16384,), generator=g, device="cuda")
    a = cuda_lib.lce_logprobs(H, W, y, top_k=3, chunk_tokens=16384)
    b = cuda_lib.lce_logprobs(H, W, y, top_k=3, chunk_tokens=2048)
    for x, z in zip(a, b):
        assert torch.equal(x, z)


# N, d, V, T, chunk
GRAD_CASES = [
    (1, 64, 37, 1.0, 0),
    (3, 72, 2, 0.7, 0),
    (129, 136, 4099, 1.0, 64),
    (129, 8, 37, 1.0, 0),
    (250, 264, 4099, 0.9, 0),
    (300, 264, 1000, 2.0, 128),
    (513, 256, 1000, 1.0, 200),
]


@pytest.mark.parametrize("N,d,V,T,chunk", GRAD_CASES)
def test_logprobs_backward(cuda_lib, N, d, V, T, chunk):
    torch = _torch()
    rng, H, W, y = make(N, d, V, seed=V + N)
    Ht, Wt = heads(H, W)
    g1, g2 = rng.standard_normal(N).astype(np.float32) / N, rng.standard_normal(N).astype(np.float32) / N
    kw = dict(temperature=T, chunk_tokens=chunk)
    logp, lse, ent, _, _ = cuda_lib.lce_logprobs(Ht, Wt, dev(y), **kw)
    dH, dW = cuda_lib.lce_logprobs_backward(Ht, Wt, dev(y), logp, lse, ent, dev(g1), dev(g2), sync_check=True, **kw)
    check_grads(dH, dW, oracle.logprobs_backward_f64(H, W, y, g1, g2, temperature=T), scaled=True)
    # one gradient at a time gives the same values
    only_H, none = cuda_lib.lce_logprobs_backward(Ht, Wt, dev(y), logp, lse, ent, dev(g1), dev(g2), need_dW=False, **kw)
    assert none is None and torch.equal(only_H, dH)
    none, only_W = cuda_lib.lce_logprobs_backward(Ht, Wt, dev(y), logp, lse, ent, dev(g1), dev(g2), need_dH=False, **kw)
    assert none is None and torch.equal(only_W, dW)
    # from logits that the forward kept; a bf16 dW
    kept = torch.empty(N, cuda_lib.lce_logits_stride(V), device="cuda")
    again = cuda_lib.lce_logprobs(Ht, Wt, dev(y), logits=kept, **kw)
    assert torch.equal(kept[:, :V].double().cpu(), torch.from_numpy(H @ W.T))
    for a, b in zip(again[:3], (logp, lse, ent)):
        close(a, np64(b), 2.0 ** -20 * (1 + np.abs(np64(b))), "with kept logits")
    for dt in (torch.float32, torch.bfloat16):
        dH2, dW2 = cuda_lib.lce_logprobs_backward(Ht, Wt, dev(y), logp, lse, ent, dev(g1), dev(g2), logits=kept, dW_dtype=dt,
                                                  **kw)
        assert torch.equal(dH2, dH) and torch.equal(dW2, dW.to(dt))
    dH2, dW2 = cuda_lib.lce_logprobs_backward(Ht, Wt, dev(y), logp, lse, ent, dev(g1), dev(g2), dW_dtype=torch.bfloat16, **kw)
    assert torch.equal(dH2, dH) and torch.equal(dW2, dW.bfloat16())
    # without the entropy's share; added to a dW that is there
    ref = oracle.logprobs_backward_f64(H, W, y, g1, None, temperature=T)
    dH, dW = cuda_lib.lce_logprobs_backward(Ht, Wt, dev(y), logp, lse, None, dev(g1), **kw)
    check_grads(dH, dW, ref, scaled=True)
    base = torch.ones(V, d, device="cuda")
    _, acc = cuda_lib.lce_logprobs_backward(Ht, Wt, dev(y), logp, lse, None, dev(g1), dW=base, accumulate_dW=True, **kw)
    # the sum with 1 rounds to fp32 once per chunk
    close(acc, 1.0 + np64(dW), 2.0 ** -23 * (1 + (N // chunk if chunk else 0)) * (1 + np.abs(np64(dW))) + 1e-7, "dW added")


@pytest.mark.parametrize("keep", [False, True])
def test_masked_rows_of_nan_have_zero_gradients(cuda_lib, keep):
    """Rows without upstream gradient (padding that holds NaN and infinities): dH is zero there and the
    other rows are not touched. (dW sums over all rows of H, as the formula does, so it is not asked for.)"""
    torch = _torch()
    rng, H, W, y = make(150, 64, 1000)
    y[:] = rng.integers(0, 1000, 150)
    Ht, Wt = heads(H, W)
    g1, g2 = rng.standard_normal(150).astype(np.float32), rng.standard_normal(150).astype(np.float32)
    masked = np.zeros(150, bool)
    masked[[3, 77, 149]] = True
    y[masked], g2[masked] = oracle.IGNORE_INDEX, 0.0
    g1[masked] = np.nan      # and its upstream gradient may be anything
    kept = torch.empty(150, 1024, device="cuda") if keep else None

    def run(h):
        logp, lse, ent, _, _ = cuda_lib.lce_logprobs(h, Wt, dev(y), logits=kept)
        return cuda_lib.lce_logprobs_backward(h, Wt, dev(y), logp, lse, ent, dev(g1), dev(g2), logits=kept, need_dW=False)[0]

    want = run(Ht)
    Ht[3], Ht[77], Ht[149, 5] = float("nan"), float("inf"), -float("inf")
    got = run(Ht)
    assert torch.equal(got, want) and not got[dev(masked)].any()


def teacher(rng, N, V, K, bf16=False):
    """Top entries with every irregularity: short lists, no list, -inf values, an index twice."""
    idx = np.stack([rng.permutation(V)[:K] if K <= V else rng.integers(0, V, K) for _ in range(N)]).astype(np.int64)
    t = (3 * rng.standard_normal((N, K))).astype(np.float32)
    if bf16:
        t = np.round(t * 8) / 8
    for i in range(N):
        what = rng.integers(0, 8)
        if what == 0:
            idx[i, rng.integers(0, K):] = oracle.IGNORE_INDEX
        elif what == 1:
            idx[i] = oracle.IGNORE_INDEX
        elif what == 2:
            t[i, rng.random(K) < 0.5] = -np.inf
        elif what == 3 and K > 1:
            idx[i, K - 1] = idx[i, 0]
            idx[i, K // 2] = idx[i, 0]
    return idx, t


# N, d, V, K, T, chunk, teacher's type
DISTILL_CASES = [
    (1, 8, 1, 1, 1.0, 0, "f32"),
    (1, 64, 37, 5, 1.0, 0, "f32"),
    (3, 72, 2, 3, 0.7, 0, "bf16"),      # more entries than words
    (129, 136, 4099, 128, 1.0, 64, "f32"),
    (129, 8, 37, 20, 2.0, 0, "bf16"),
    (300, 264, 1001, 33, 3.0, 128, "f32"),
    (513, 256, 1000, 1, 1.0, 200, "bf16"),
    (40, 64, 30011, 64, 1.0, 0, "f32"),
]


@pytest.mark.parametrize("N,d,V,K,T,chunk,kind", DISTILL_CASES)
@pytest.mark.parametrize("renormalize", [True, False])
def test_distill(cuda_lib, N, d, V, K, T, chunk, kind, renormalize):
    torch = _torch()
    rng, H, W, _ = make(N, d, V, seed=V + K)
    idx, t = teacher(rng, N, V, K, kind == "bf16")
    if not renormalize:
        T, t = 1.0, t - 8
    Ht, Wt, it = *heads(H, W), dev(idx)
    tt = dev(t, torch.bfloat16 if kind == "bf16" else torch.float32)
    kw = dict(temperature=T, renormalize=renormalize, chunk_tokens=chunk)
    g = dev(np.array([1.5], np.float32))
    loss, row, dH, dW = cuda_lib.lce_distill_fwd_bwd(Ht, Wt, it, tt, g, sync_check=True, **kw)
    ref = oracle.distill_f64(H, W, idx, np64(tt), temperature=T, renormalize=renormalize, grad_loss=1.5)
    # row_loss = T^2 sum q (log q - logp): |log q| errs like lse (exponentials and sums of the same kind)
    lse = oracle.logprobs_f64(H, W, np.zeros(N, np.int64), temperature=T)["lse"]
    mass = oracle.teacher_f64(idx, np64(tt), V, temperature=T, renormalize=renormalize)[0].sum(axis=1)
    tol = T * T * (mass + 1e-3) * (4 * tol_lse(H, W, lse, T) + 2.0 ** -20 * (16 + np.abs(t[np.isfinite(t)]).max(initial=0)))
    close(row, ref["row_loss"], tol, "row_loss")
    close(loss, ref["loss"], tol.mean() * N / max(1, (mass > 0).sum()), "loss")
    check_grads(dH, dW, ref)
    assert not dH[dev(mass == 0)].any()
    narrow = cuda_lib.lce_distill_fwd_bwd(Ht, Wt, it, tt, g, dW_dtype=torch.bfloat16, **kw)
    assert torch.equal(narrow[2], dH) and torch.equal(narrow[3], dW.bfloat16())
    loss2, row2 = cuda_lib.lce_distill_forward(Ht, Wt, it, tt, **kw)
    assert torch.equal(loss2, loss) and torch.equal(row2, row)
    only_H = cuda_lib.lce_distill_fwd_bwd(Ht, Wt, it, tt, g, need_dW=False, **kw)
    assert only_H[3] is None and torch.equal(only_H[2], dH)
    only_W = cuda_lib.lce_distill_fwd_bwd(Ht, Wt, it, tt, g, need_dH=False, **kw)
    assert only_W[2] is None and torch.equal(only_W[3], dW)


def test_distill_sum_override_and_accumulation(cuda_lib):
    torch = _torch()
    rng, H, W, _ = make(200, 64, 500)
    idx, t = teacher(rng, 200, 500, 6)
    Ht, Wt, it, tt = *heads(H, W), dev(idx), dev(t)
    ref = oracle.distill_f64(H, W, idx, t, reduction=oracle.SUM)
    loss, _, dH, dW = cuda_lib.lce_distill_fwd_bwd(Ht, Wt, it, tt, reduction="sum")
    assert abs(loss.item() - ref["loss"]) <= 1e-5 * abs(ref["loss"])
    check_grads(dH, dW, ref)
    ref = oracle.distill_f64(H, W, idx, t, n_valid_override=1000)
    half = [cuda_lib.lce_distill_fwd_bwd(Ht[s], Wt, it[s], tt[s], n_valid_override=1000) for s in
            (slice(0, 100), slice(100, 200))]
    assert abs(sum(x[0].item() for x in half) - ref["loss"]) <= 1e-5 * abs(ref["loss"])
    acc = half[0][3].clone()
    cuda_lib.lce_distill_fwd_bwd(Ht[100:], Wt, it[100:], tt[100:], n_valid_override=1000, dW=acc, accumulate_dW=True)
    check_grads(torch.cat([half[0][2], half[1][2]]), acc, ref)


def test_distill_all_rows_empty_and_bad_index(cuda_lib):
    torch = _torch()
    rng, H, W, _ = make(70, 64, 500)
    Ht, Wt = heads(H, W)
    idx = torch.full((70, 5), -100, device="cuda")
    t = torch.zeros(70, 5, device="cuda")
    loss, row, dH, dW = cuda_lib.lce_distill_fwd_bwd(Ht, Wt, idx, t, sync_check=True)
    assert loss.item() == 0 and not row.any() and not dH.any() and not dW.any()
    idx[:, :2] = torch.tensor([3, 9], device="cuda")
    want = cuda_lib.lce_distill_fwd_bwd(Ht, Wt, idx, t)
    idx[5, 3], idx[6, 4] = 500, -7        # not kept, and told
    with pytest.raises(cuda_lib.LCEError) as err:
        cuda_lib.lce_distill_fwd_bwd(Ht, Wt, idx, t, sync_check=True)
    assert err.value.code == cuda_lib.LCE_ERR_LABEL_RANGE
    for a, b in zip(cuda_lib.lce_distill_fwd_bwd(Ht, Wt, idx, t), want):
        assert torch.equal(a, b)


def test_teacher_to_student(cuda_lib):
    """The teacher's alternatives are the student's targets; a student equal to
    its teacher, every word kept, has no loss and (to rounding) no gradient."""
    torch = _torch()
    rng, H, W, y = make(150, 64, 2000, seed=1)
    _, H2, W2, _ = make(150, 128, 2000, seed=2)
    teacher_H, teacher_W = heads(H, W)
    student_H, student_W = heads(H2, W2)
    _, _, _, tl, ti = cuda_lib.lce_logprobs(teacher_H, teacher_W, dev(y), top_k=24)
    loss, row, dH, dW = cuda_lib.lce_distill_fwd_bwd(student_H, student_W, ti, tl, renormalize=False)
    ref = oracle.distill_f64(H2, W2, ti.cpu().numpy(), np64(tl), renormalize=False)
    assert abs(loss.item() - ref["loss"]) <= 1e-5 * abs(ref["loss"])
    check_grads(dH, dW, ref)
    small = teacher_W[:100]
    _, _, _, tl, ti = cuda_lib.lce_logprobs(teacher_H, small, dev(np.zeros(150, np.int64)), top_k=100)
    loss, row, dH, dW = cuda_lib.lce_distill_fwd_bwd(teacher_H, small, ti, tl, renormalize=False)
    assert abs(loss.item()) < 2.0 ** -14
    assert dH.float().abs().max().item() < 1e-5


@pytest.mark.parametrize("N,d,V,chunk", [(6500, 2048, 151936, 0), (700, 7168, 151655, 512)])
def test_full_heads_sampled(cuda_lib, N, d, V, chunk):
    """The heads' real sizes, two chunks: rows of both sides of the chunk boundary and of both ends, and
    vocabulary rows of the tails, against the definition in fp64."""
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(N)
    sigma = 0.02 if d <= 2048 else 0.01
    W = (torch.randn(V, d, generator=g, device="cuda") * (sigma * 1024)).round().clamp(-127, 127).div(1024).bfloat16()
    y = torch.randint(0, V, (N,), generator=g, device="cuda")
    H = torch.randn(N, d, generator=g, device="cuda")
    H += W[y].float() * (14.0 * torch.rand(N, 1, generator=g, device="cuda") / (sigma * sigma * d))
    H = (H * 16).round().clamp(-127, 127).div(16).bfloat16()
    y[::17] = oracle.IGNORE_INDEX
    edge = chunk or 3328   # equal chunks by default: ceil(6500 / 2) in whole tiles
    rows = np.array([0, 1, edge - 1, edge, edge + 1, N // 3, N - 2, N - 1])
    cols = np.array([0, 127, 128, 255, 256, V // 2, V - 130, V - 2, V - 1])
    Hn, Wn, yn = np64(H), np64(W), y.cpu().numpy()
    out = cuda_lib.lce_logprobs(H, W, y, top_k=20, chunk_tokens=chunk, sync_check=True)
    logp, lse, ent = out[:3]
    check_scores([x[torch.from_numpy(rows).cuda()] for x in out], Hn[rows], Wn, yn[rows], 1.0, 20)
    a = torch.randn(N, generator=g, device="cuda")
    e = 0.1 * torch.randn(N, generator=g, device="cuda")
    dH, dW = cuda_lib.lce_logprobs_backward(H, W, y, logp, lse, ent, a, e, chunk_tokens=chunk)
    part = oracle.logprobs_backward_f64(Hn[rows], Wn, yn[rows], np64(a)[rows], np64(e)[rows])
    check_grads(dH[torch.from_numpy(rows).cuda()], None, part)

    def sampled_dW(G, size, got, scaled):   # columns of G [N, cols] in fp64 from the call's lse
        check_grads(None, got[torch.from_numpy(cols).cuda()],
                    {"dW": G.T @ Hn, "dW_bulk": size.T @ np.abs(Hn)}, scaled=scaled)

    logq = Hn @ Wn[cols].T - np64(lse)[:, None]
    p, hot = np.exp(logq), (yn[:, None] == cols[None, :]).astype(float)
    an = np.where(yn >= 0, np64(a), 0.0)[:, None]
    dev_ = np64(e)[:, None] * (logq + np64(ent)[:, None])
    sampled_dW(hot * an - p * (an + dev_), hot * np.abs(an) + p * (np.abs(an) + np.abs(dev_)), dW, True)
    # distillation from these alternatives
    idx, t = out[4].clone(), out[3]
    idx[5::11, 7:] = oracle.IGNORE_INDEX
    idx[3::13] = oracle.IGNORE_INDEX
    idx[:9, 0] = torch.from_numpy(cols).cuda()
    loss, row, dH, dW = cuda_lib.lce_distill_fwd_bwd(H, W, idx, t, renormalize=False, chunk_tokens=chunk,
                                                     sync_check=True)
    n = int((idx >= 0).any(1).sum())
    part = oracle.distill_f64(Hn[rows], Wn, idx.cpu().numpy()[rows], np64(t)[rows], renormalize=False,
                              n_valid_override=n)
    close(row[torch.from_numpy(rows).cuda()], part["row_loss"], 2.0 ** -14, "row_loss")
    check_grads(dH[torch.from_numpy(rows).cuda()], None, part)
    assert abs(loss.item() - row.double().sum().item() / n) <= 2.0 ** -22 * abs(loss.item())
    q = np.where(idx.cpu().numpy() >= 0, np.exp(np64(t)), 0.0)
    hot = np.stack([np.where(idx.cpu().numpy() == c, q, 0.0).sum(1) for c in cols], axis=1)
    mass = q.sum(1, keepdims=True)
    sampled_dW((mass * p - hot) / n, (mass * p + hot) / n, dW, False)


# --------------------------------------------------------------------------- as programs use them
def test_autograd_modules(cuda_lib):
    torch = _torch()
    from chunked_lm_head_linear_gb300.autograd import FusedLinearDistillation, FusedLinearLogProbs
    rng, H, W, y = make(200, 64, 700)
    Ht, Wt = heads(H, W)
    Ht.requires_grad_(True)
    Wt.requires_grad_(True)
    w = dev(rng.standard_normal(200).astype(np.float32))
    logp, ent = FusedLinearLogProbs(temperature=0.8)(Ht, Wt, dev(y))
    dH, dW = torch.autograd.grad((logp * w).sum() - 0.5 * ent.sum(), [Ht, Wt])
    assert dH.dtype == dW.dtype == torch.bfloat16
    ref = oracle.logprobs_backward_f64(H, W, y, np64(w), np.full(200, -0.5), temperature=0.8)
    check_grads(dH, dW, ref, scaled=True)
    for recompute in (True, False):   # the same from recomputed and from kept logits
        logp, ent = FusedLinearLogProbs(temperature=0.8, recompute=recompute, chunk_tokens=96)(Ht, Wt, dev(y))
        a, b = torch.autograd.grad((logp * w).sum() - 0.5 * ent.sum(), [Ht, Wt])
        check_grads(a, b, ref, scaled=True)
    # outputs used alone; a frozen head
    logp, ent = FusedLinearLogProbs()(Ht, Wt.detach(), dev(y))
    check_grads(torch.autograd.grad(logp.sum(), Ht)[0], None,
                oracle.logprobs_backward_f64(H, W, y, np.ones(200), None))
    logp, ent = FusedLinearLogProbs()(Ht, Wt, dev(y))
    check_grads(torch.autograd.grad(ent.sum(), Ht)[0], None,
                oracle.logprobs_backward_f64(H, W, y, np.zeros(200), np.ones(200)))
    idx, t = teacher(rng, 200, 700, 9)
    kd = FusedLinearDistillation(temperature=2.0)
    loss = kd(Ht, Wt, dev(idx), dev(t))
    assert loss.shape == ()
    dH, dW = torch.autograd.grad(3.0 * loss, [Ht, Wt], retain_graph=True)
    ref = oracle.distill_f64(H, W, idx, t, temperature=2.0, grad_loss=3.0)
    # scaled after their rounding: one rounding more
    for got, name in ((dH, "dH"), (dW, "dW")):
        assert got.dtype == torch.bfloat16
        close(got, ref[name], (U + 2.0 ** -10) * ref[name + "_bulk"] + 2.01 * U * np.abs(ref[name]) + 1e-30, name)
    with pytest.raises(RuntimeError, match="run the forward again"):
        torch.autograd.grad(loss, [Ht, Wt])
    with torch.no_grad():
        assert torch.equal(kd(Ht, Wt, dev(idx), dev(t)), loss)
    # one side frozen; a loss scale that is a power of two rounds nothing
    for h, w_, k in ((Ht, Wt.detach(), 0), (Ht.detach(), Wt, 1)):
        got, = torch.autograd.grad(1024.0 * kd(h, w_, dev(idx), dev(t)), (h, w_)[k])
        want = oracle.distill_f64(H, W, idx, t, temperature=2.0, grad_loss=1024.0)
        check_grads(got if k == 0 else None, got if k == 1 else None, want)
    # no tokens
    none = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    dH, dW = torch.autograd.grad(kd(none, Wt, dev(idx[:0]), dev(t[:0])), [none, Wt])
    assert dH.shape == (0, 64) and not dW.any()
    logp, ent = FusedLinearLogProbs()(none, Wt, dev(y[:0]))
    dH, dW = torch.autograd.grad(logp.sum() + ent.sum(), [none, Wt])
    assert dH.shape == (0, 64) and not dW.any()


@pytest.mark.parametrize("N", [8, 300])
def test_streams_graphs_and_a_shared_workspace(cuda_lib, N):
    """Calls on a side stream, captured once and replayed on new inputs; two captured
    graphs that share a workspace, replayed one after the other."""
    torch = _torch()
    rng, H, W, y = make(N, 64, 3001)
    _, H2, _, _ = make(N, 64, 3001, seed=9)
    idx, t = teacher(rng, N, 3001, 7)
    Ht, Wt = heads(H, W)
    other, yt, it, tt = dev(H2, torch.bfloat16), dev(y), dev(idx), dev(t)
    g1 = dev(rng.standard_normal(N).astype(np.float32))
    need = max(cuda_lib.lce_logprobs_workspace_size(N, 64, 3001, 5), cuda_lib.lce_logprobs_backward_workspace_size(N, 64, 3001),
               cuda_lib.lce_distill_workspace_size(N, 64, 3001, 7, True))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def score(h):
        out = cuda_lib.lce_logprobs(h, Wt, yt, top_k=5, workspace=ws)
        return list(out) + list(cuda_lib.lce_logprobs_backward(h, Wt, yt, out[0], out[1], out[2], g1, g1, workspace=ws))

    def kd(h):
        return list(cuda_lib.lce_distill_fwd_bwd(h, Wt, it, tt, workspace=ws))

    want = [[score(h), kd(h)] for h in (Ht, other)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [score(Ht), kd(Ht)]
    side.synchronize()
    for a, b in zip(got[0] + got[1], want[0][0] + want[0][1]):
        assert torch.equal(a, b)
    x = Ht.clone()
    graphs, outs = [], []
    for f in (score, kd):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(f(x))
        graphs.append(graph)
    for k, h in ((1, other), (0, Ht), (1, other)):
        x.copy_(h)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs[0] + outs[1], want[k][0] + want[k][1]):
            assert torch.equal(a, b)


def test_autograd_captured_and_replayed(cuda_lib):
    """A training step of both modules, forward and torch.autograd.grad, captured once and replayed on new
    hidden states."""
    torch = _torch()
    from chunked_lm_head_linear_gb300.autograd import FusedLinearDistillation, FusedLinearLogProbs
    rng, H, W, y = make(200, 1024, 700)
    idx, t = teacher(rng, 200, 700, 9)
    Ht, Wt = heads(H, W)
    it, tt, yt = dev(idx), dev(t), dev(y)
    g = dev(rng.standard_normal(200).astype(np.float32))
    x, w = Ht.clone().requires_grad_(True), Wt.clone().requires_grad_(True)

    def step():
        logp, ent = FusedLinearLogProbs()(x, w, yt)
        loss = FusedLinearDistillation()(x, w, it, tt)
        return [logp, ent, loss, *torch.autograd.grad([logp, ent], [x, w], [g, g]), *torch.autograd.grad(loss, [x, w])]

    want = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for k in range(2):
            with torch.no_grad():
                x.copy_(Ht if k == 0 else -Ht)
            want.append([o.detach().clone() for o in step()])
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in (0, 1, 0):
        with torch.no_grad():
            x.copy_(Ht if k == 0 else -Ht)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want[k]):
            assert torch.equal(a, b)


def test_two_streams_at_once(cuda_lib):
    """Calls whose work overlaps on the GPU, each with its own workspace and the stream argument."""
    torch = _torch()
    rng, H, W, y = make(700, 256, 5000)
    idx, t = teacher(rng, 700, 5000, 12)
    Ht, Wt, yt, it, tt = *heads(H, W), dev(y), dev(idx), dev(t)
    want = [cuda_lib.lce_logprobs(Ht, Wt, yt, top_k=9), cuda_lib.lce_logprobs(Ht[:5], Wt, yt[:5], top_k=9),
            cuda_lib.lce_distill_fwd_bwd(Ht, Wt, it, tt)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        got = [cuda_lib.lce_logprobs(Ht, Wt, yt, top_k=9, stream=streams[0]),
               cuda_lib.lce_logprobs(Ht[:5], Wt, yt[:5], top_k=9, stream=streams[1]),
               cuda_lib.lce_distill_fwd_bwd(Ht, Wt, it, tt, stream=streams[2])]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for x, z in zip(a, b):
                assert torch.equal(x, z)


def test_caller_tensors_are_checked(cuda_lib):
    torch = _torch()
    _, H, W, y = make(20, 64, 300)
    Ht, Wt, yt = *heads(H, W), dev(y)
    f = torch.zeros(20, device="cuda")
    idx = torch.zeros(20, 4, dtype=torch.int64, device="cuda")
    t = torch.zeros(20, 4, device="cuda")
    for call in (lambda: cuda_lib.lce_logprobs(Ht.float(), Wt, yt), lambda: cuda_lib.lce_logprobs(Ht.t(), Wt, yt),
                 lambda: cuda_lib.lce_logprobs(Ht, Wt, yt.int()),
                 lambda: cuda_lib.lce_logprobs_backward(Ht, Wt, yt, f, f[:5], f, f),
                 lambda: cuda_lib.lce_logprobs_backward(Ht, Wt, yt, f, f, None, f, f),
                 lambda: cuda_lib.lce_logprobs_backward(Ht, Wt, yt, f, f, f, f.double()),
                 lambda: cuda_lib.lce_logprobs_backward(Ht, Wt, yt, f, f, f, f, need_dH=False, need_dW=False),
                 lambda: cuda_lib.lce_logprobs_backward(Ht, Wt, yt, f, f, f, f, accumulate_dW=True),
                 lambda: cuda_lib.lce_distill_forward(Ht, Wt, idx.int(), t),
                 lambda: cuda_lib.lce_distill_forward(Ht, Wt, idx, t.half()),
                 lambda: cuda_lib.lce_distill_forward(Ht, Wt, idx, t[:, :3]),
                 lambda: cuda_lib.lce_distill_forward(Ht, Wt, idx[:, ::2], t[:, ::2]),
                 lambda: cuda_lib.lce_distill_forward(Ht, Wt, idx, t, temperature=2.0, renormalize=False)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: cuda_lib.lce_logprobs(Ht, Wt, yt, top_k=301), lambda: cuda_lib.lce_logprobs(Ht, Wt, yt, top_k=-1),
                 lambda: cuda_lib.lce_logprobs(Ht, Wt, yt, temperature=0.0)):
        with pytest.raises(cuda_lib.LCEError) as err:
            call()
        assert err.value.code == cuda_lib.LCE_ERR_INVALID_ARG
    with pytest.raises(cuda_lib.LCEError) as err:
        cuda_lib.lce_logprobs(Ht, Wt, yt, top_k=3, workspace=torch.empty(1000, dtype=torch.uint8, device="cuda"))
    assert err.value.code == cuda_lib.LCE_ERR_WORKSPACE
    auto = cuda_lib.lce_logprobs(Ht, Wt, yt, top_k=3, chunk_tokens="auto")
    for a, b in zip(auto, cuda_lib.lce_logprobs(Ht, Wt, yt, top_k=3)):
        assert torch.equal(a, b)


# --------------------------------------------------------------------------- cold, confident and masked rows
@pytest.mark.parametrize("N", [5, 130])
@pytest.mark.parametrize("T", [1e-6, 1e-4])
def test_logprobs_of_large_logits_at_low_temperatures(cuda_lib, N, T):
    """Logits of up to 7000 of either sign, ties among them, over temperatures that make them 7e9. z - max is exact,
    so log-probabilities err by the roundings of 1 / T, the product and the last sum, 3 eps of themselves,
    and by what lse - max / T errs by, below 2^-16 (13 times that in the entropy)."""
    V, d = 3000, 512
    rng = np.random.default_rng(N)
    W = np.full((V, d), 1.5)
    W[:, 64:] = grid(rng.standard_normal((V, 1)) / 8 + 1.25, 64)
    H = np.repeat(rng.integers(60, 121, (N, 1)) / 16 * rng.choice([-1.0, 1.0], (N, 1)), d, axis=1)
    y = rng.integers(0, V, N)
    T = float(np.float32(T))
    Ht, Wt, yt = *heads(H, W), dev(y)
    assert np.abs(H @ W.T).max() > 4000
    logp, lse, ent, tl, ti = cuda_lib.lce_logprobs(Ht, Wt, yt, top_k=9, temperature=T)
    ref = oracle.logprobs_f64(H, W, y, temperature=T, top_k=9)
    assert (ti.cpu().numpy() == ref["top_idx"]).all()
    for got, name, part in ((logp, "logp", 1.0), (tl, "top_logp", 1.0), (lse, "lse", 1.0), (ent, "entropy", 13.0)):
        assert np.isfinite(np64(got)).all(), name
        close(got, ref[name], part * 2.0 ** -16 + 2.0 ** -22 * np.abs(ref[name]), name)
    idx, t = ti, (tl * 0.0).contiguous()
    loss, row = cuda_lib.lce_distill_forward(Ht, Wt, idx, t, temperature=T)
    want = oracle.distill_f64(H, W, ref["top_idx"], np.zeros((N, 9)), temperature=T)
    # T^2 (log q - mean of nine log-probabilities)
    close(row, want["row_loss"], T * T * (2.0 ** -15 + 2.0 ** -21 * np.abs(ref["top_logp"]).max(axis=1)), "row_loss")


def near_ties(N, T, seed=0, boost=1.0):
    """Rows whose largest logits, boost * 16 to 31, lie a few steps of boost * 2^-18 apart or are equal: a
    distribution over many words however low the temperature. Exact in fp32 in any order of the sum
    (whole multiples of boost * 2^-18 below boost * 64). The words' other features meet zeros of H."""
    rng = np.random.default_rng(seed)
    V, d = 700, 64
    W = grid(rng.standard_normal((V, d)), 64)
    W[:, 0] = np.where(np.arange(V) % 2 == 0, 8.0, rng.integers(-32, 31, V) / 4)
    W[:, 1] = rng.integers(0, 64, V) * 2.0 ** -18
    H = np.zeros((N, d))
    H[:, 0] = 2 + rng.integers(0, 31, N) / 16
    H[:, 1] = 1.0
    y = 2 * rng.integers(0, V // 2, N)
    y[::7] += 1                          # an unlikely label
    y[3::11] = oracle.IGNORE_INDEX
    return rng, H * boost, W, y, float(np.float32(T * boost))


def with_underflow(ref, H, W, T):
    """The bounds of check_grads with what fp32 cannot hold. An entry of G is p c with |c| <= (|a| + |e| (|log p|
    + entropy)) / T. p below 2^-126 may be 0, where |log p| is 88 (p |log p| only falls with p), the entropy
    below 7 and |a|, |e| below 5: 2^-126 5 96 / T < 2^-117 / T is lost; as much again where the entry over its
    row's scale, itself at most such a c, is below 2^-126. Sums over rows and words follow."""
    lost = 2.0 ** -116 / T / U      # the bounds take at least U of the bulk
    return dict(ref, dH_bulk=ref["dH_bulk"] + lost * np.abs(W).sum(axis=0),
                dW_bulk=ref["dW_bulk"] + lost * np.abs(H).sum(axis=0))


COLD = [1.0, 1e-2, 1e-3, 1e-4, 1e-5, 1e-6]


@pytest.mark.parametrize("N", [5, 130])
@pytest.mark.parametrize("T", COLD)
def test_gradients_at_low_temperatures(cuda_lib, N, T):
    """p does not lose what z / T is rounded by: logits of 20 to 30 with near-ties, down to the coldest
    temperature, recomputed and kept. The bounds are those of ordinary temperatures: with exact logits
    the exponents (z - max) / T err by 2^-23 of themselves only."""
    torch = _torch()
    rng, H, W, y, T = near_ties(N, T, seed=N)
    Ht, Wt, yt = *heads(H, W), dev(y)
    g1, g2 = rng.standard_normal(N).astype(np.float32), rng.standard_normal(N).astype(np.float32)
    ref = oracle.logprobs_backward_f64(H, W, y, g1, g2, temperature=T)
    ref = with_underflow(ref, H, W, T)
    kept = torch.empty(N, cuda_lib.lce_logits_stride(len(W)), device="cuda")
    logp, lse, ent, _, _ = cuda_lib.lce_logprobs(Ht, Wt, yt, temperature=T, logits=kept)
    for logits in (None, kept):
        dH, dW = cuda_lib.lce_logprobs_backward(Ht, Wt, yt, logp, lse, ent, dev(g1), dev(g2), temperature=T,
                                                logits=logits)
        check_grads(dH, dW, ref, scaled=True)


@pytest.mark.parametrize("N", [5, 130])
@pytest.mark.parametrize("T,boost", [(t, 1.0) for t in COLD] + [(2.0 ** -15, 2.0 ** 15), (1e-4, 2.0 ** 17)])
def test_autograd_at_low_temperatures_and_large_logits(cuda_lib, N, T, boost):
    """The same through the module, and with logits of up to 2^22 at temperatures near 1."""
    torch = _torch()
    from chunked_lm_head_linear_gb300.autograd import FusedLinearLogProbs
    rng, H, W, y, T = near_ties(N, T, seed=N + 1, boost=boost)
    Ht, Wt = (x.requires_grad_(True) for x in heads(H, W))
    g = [dev(rng.standard_normal(N).astype(np.float32)) for _ in range(2)]
    ref = oracle.logprobs_backward_f64(H, W, y, np64(g[0]), np64(g[1]), temperature=T)
    ref = with_underflow(ref, H, W, T)
    for recompute in (True, False):
        out = FusedLinearLogProbs(temperature=T, recompute=recompute, chunk_tokens=100)(Ht, Wt, dev(y))
        dH, dW = torch.autograd.grad(out, [Ht, Wt], g)
        check_grads(dH, dW, ref, scaled=True)


@pytest.mark.parametrize("N", [12, 200])
def test_entropy_gradient_of_confident_rows(cuda_lib, N):
    """One token has nearly all of p: log p + entropy is of the size of 1 - p there, and so is every entry
    of G. Both keep their relative precision (2^-15, see the log-probabilities near zero; their sum is
    20 to 30 times each, positive), so that no absolute error stays: the bound is the relative one alone."""
    torch = _torch()
    from chunked_lm_head_linear_gb300.autograd import FusedLinearLogProbs
    V, d, label = 5000, 64, 1234
    rng = np.random.default_rng(5)
    W = grid(rng.standard_normal((V, d)), 64)
    W[:, 0] = -1.0
    W[label, 0] = 0.0
    W[:, 1] = rng.integers(-8, 9, V) / 64
    H = np.zeros((N, d))
    H[:, 0] = 20 + np.arange(N) % 10
    H[:, 1] = 1.0
    y = np.where(np.arange(N) % 3 < 2, 77, label)
    Ht, Wt = (x.requires_grad_(True) for x in heads(H, W))
    g = rng.standard_normal(N).astype(np.float32)
    ref = oracle.logprobs_backward_f64(H, W, y, np.zeros(N), g)
    ref = {k: v for k, v in ref.items() if not k.endswith("_slack")}
    for recompute in (True, False):
        _, ent = FusedLinearLogProbs(recompute=recompute)(Ht, Wt, dev(y))
        dH, dW = torch.autograd.grad(ent, [Ht, Wt], dev(g))
        check_grads(dH, dW, ref, scaled=True)


def _cold_child():
    """The backward that computes the rows' statistics itself, and the one that is given them, on the
    bounds-checking build."""
    import torch

    from chunked_lm_head_linear_gb300 import build, lce
    lce.load(build.build(checks=True))
    for N, chunk in [(1, 0), (96, 0), (130, 0), (300, 100)]:
        rng, H, W, y, T = near_ties(N, 1e-4, seed=N)
        Ht, Wt, yt = *heads(H, W), dev(y)
        g = dev(rng.standard_normal(N).astype(np.float32))
        ref = oracle.logprobs_backward_f64(H, W, y, np64(g), np64(g), temperature=T)
        ref = with_underflow(ref, H, W, T)
        kept = torch.empty(N, lce.lce_logits_stride(len(W)), device="cuda")
        for logits in (None, kept):
            kw = dict(temperature=T, chunk_tokens=chunk, logits=logits, sync_check=True)
            logp, lse, ent, _, _, stats = lce.lce_logprobs_keep(Ht, Wt, yt, **kw)
            check_grads(*lce.lce_logprobs_keep_backward(Ht, Wt, yt, logp, stats, ent, g, g, **kw), ref, scaled=True)
            check_grads(*lce.lce_logprobs_backward(Ht, Wt, yt, logp, lse, ent, g, g, **kw), ref, scaled=True)
    print("checked build: ok")


def test_bounds_checking_build_at_a_low_temperature(cuda_lib):
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([os.path.dirname(here), here]))
    r = subprocess.run([sys.executable, "-c", "import test_tokens_gpu as t; t._cold_child()"], env=env, cwd=here,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "checked build: ok" in r.stdout, (r.stdout + r.stderr)[-3000:]


def test_cold_backward_tells_of_labels_and_captures(cuda_lib):
    """The statistics pass leaves the status bits to the call: a label out of range is told and has no
    gradient; and the call can be captured and replayed."""
    torch = _torch()
    rng, H, W, y, T = near_ties(130, 1e-4)
    Ht, Wt, yt = *heads(H, W), dev(y)
    g = dev(rng.standard_normal(130).astype(np.float32))
    kw = dict(temperature=T, chunk_tokens=50)
    logp, lse, ent, _, _ = cuda_lib.lce_logprobs(Ht, Wt, yt, **kw)
    yt[3] = oracle.IGNORE_INDEX
    want = cuda_lib.lce_logprobs_backward(Ht, Wt, yt, logp, lse, ent, g, g, **kw)
    yt[3] = 700
    with pytest.raises(cuda_lib.LCEError) as err:
        cuda_lib.lce_logprobs_backward(Ht, Wt, yt, logp, lse, ent, g, g, sync_check=True, **kw)
    assert err.value.code == cuda_lib.LCE_ERR_LABEL_RANGE
    for a, b in zip(cuda_lib.lce_logprobs_backward(Ht, Wt, yt, logp, lse, ent, g, g, **kw), want):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cuda_lib.lce_logprobs_backward(Ht, Wt, yt, logp, lse, ent, g, g, **kw)
    for x in out:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)


def _memory_case():
    """Trainable inputs of both modules: 60 MB of logits, 6 MB of dW."""
    torch = _torch()
    N, V = 300, 50000
    rng, H, W, y = make(N, 64, V)
    Ht, Wt = (x.requires_grad_(True) for x in heads(H, W))
    return (N, V, Ht, Wt, dev(y), dev(rng.integers(0, V, (N, 5))), dev(rng.standard_normal((N, 5)).astype(np.float32)),
            torch.ones(N, device="cuda"))


def test_no_grad_keeps_and_computes_nothing_for_a_backward(cuda_lib):
    torch = _torch()
    from chunked_lm_head_linear_gb300.autograd import FusedLinearDistillation, FusedLinearLogProbs
    N, V, Ht, Wt, yt, idx, t, _ = _memory_case()
    mod, kd = FusedLinearLogProbs(recompute=False), FusedLinearDistillation()
    want = [x.detach() for x in (*mod(Ht, Wt, yt), kd(Ht, Wt, idx, t))]
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            for call, need in ((lambda: mod(Ht, Wt, yt), cuda_lib.lce_logprobs_workspace_size(N, 64, V)),
                               (lambda: (kd(Ht, Wt, idx, t),), cuda_lib.lce_distill_workspace_size(N, 64, V, 5, False))):
                torch.cuda.synchronize()
                torch.cuda.reset_peak_memory_stats()
                before = torch.cuda.memory_allocated()
                got = call()
                # the forward's workspace and its few results; memory is handed out in blocks of up to 2 MB
                assert torch.cuda.max_memory_allocated() - before < need + (1 << 21)
                assert not any(x.requires_grad for x in got)
                for a, b in zip(got, want[:2] if len(got) == 2 else want[2:]):
                    assert torch.equal(a, b) if len(got) == 1 else (a - b).abs().max() < 2.0 ** -14


def test_kept_logits_are_freed_by_the_backward(cuda_lib):
    """After a backward that does not retain the graph nothing of the call is held but its outputs."""
    import gc
    torch = _torch()
    from chunked_lm_head_linear_gb300.autograd import FusedLinearLogProbs
    N, V, Ht, Wt, yt, _, _, w = _memory_case()
    mod = FusedLinearLogProbs(recompute=False)
    gc.collect()
    torch.cuda.synchronize()
    base = torch.cuda.memory_allocated()
    logp, ent = mod(Ht, Wt, yt)
    assert torch.cuda.memory_allocated() - base > 4 * N * V           # the logits wait for the backward
    want = torch.autograd.grad(logp, [Ht, Wt], w, retain_graph=True)
    got = torch.autograd.grad(logp, [Ht, Wt], w)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del want, got
    assert torch.cuda.memory_allocated() - base < 1 << 16             # logp and entropy are still here
    with pytest.raises(RuntimeError):
        torch.autograd.grad(logp, [Ht, Wt], w)
    # saved-tensor hooks see them
    seen = []
    with torch.autograd.graph.saved_tensors_hooks(lambda x: seen.append(x.numel()) or x, lambda x: x):
        mod(Ht, Wt, yt)
    assert N * cuda_lib.lce_logits_stride(V) in seen


@pytest.mark.parametrize("keep", [False, True])
def test_masked_rows_of_nan_leave_dW_alone(cuda_lib, keep):
    """Rows without upstream gradient have no share of dW either, whatever their hidden states hold."""
    torch = _torch()
    rng, H, W, y = make(150, 64, 1000)
    y[:] = rng.integers(0, 1000, 150)
    Ht, Wt = heads(H, W)
    g1, g2 = rng.standard_normal(150).astype(np.float32), rng.standard_normal(150).astype(np.float32)
    masked = np.zeros(150, bool)
    masked[[3, 77, 149]] = True
    y[masked], g2[masked] = oracle.IGNORE_INDEX, 0.0
    kept = torch.empty(150, 1024, device="cuda") if keep else None

    def run(h, **kw):
        logp, lse, ent, _, _ = cuda_lib.lce_logprobs(h, Wt, dev(y), logits=kept, chunk_tokens=100)
        return cuda_lib.lce_logprobs_backward(h, Wt, dev(y), logp, lse, ent, dev(g1), dev(g2), logits=kept,
                                              chunk_tokens=100, **kw)

    for dtype in (torch.float32, torch.bfloat16):
        want = run(Ht, dW_dtype=dtype)
        nan = Ht.clone()
        nan[3], nan[77], nan[149, 5] = float("nan"), float("inf"), -float("inf")
        for a, b in zip(run(nan, dW_dtype=dtype), want):
            assert torch.equal(a, b)


def test_distill_rows_without_a_teacher_may_hold_nan(cuda_lib):
    """Rows that keep no entry have no share of the loss, dH or dW, whatever their hidden states hold."""
    torch = _torch()
    rng, H, W, _ = make(150, 72, 500)
    idx, t = teacher(rng, 150, 500, 6)
    Ht, Wt = heads(H, W)
    idx[3], t[77] = oracle.IGNORE_INDEX, -np.inf
    idx[149] = oracle.IGNORE_INDEX
    it, tt = dev(idx), dev(t)
    nan = Ht.clone()
    nan[3], nan[77], nan[149, 5] = float("nan"), float("inf"), -float("inf")
    for kw in (dict(), dict(chunk_tokens=100), dict(dW_dtype=torch.bfloat16, chunk_tokens=64), dict(need_dH=False)):
        want = cuda_lib.lce_distill_fwd_bwd(Ht, Wt, it, tt, **kw)
        for a, b in zip(cuda_lib.lce_distill_fwd_bwd(nan, Wt, it, tt, **kw), want):
            assert a is b is None or torch.equal(a, b)


def test_kept_logits_captured_and_replayed(cuda_lib):
    """The module's step with kept logits and statistics, captured once and replayed on other hidden states."""
    torch = _torch()
    from chunked_lm_head_linear_gb300.autograd import FusedLinearLogProbs
    rng, H, W, y = make(100, 64, 700)
    Ht, Wt = heads(H, W)
    yt, g = dev(y), dev(rng.standard_normal(100).astype(np.float32))
    x, w = Ht.clone().requires_grad_(True), Wt.clone().requires_grad_(True)

    def step():
        out = FusedLinearLogProbs(recompute=False, temperature=0.01)(x, w, yt)
        return [*out, *torch.autograd.grad(out, [x, w], [g, g])]

    want = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for h in (Ht, -Ht):
            with torch.no_grad():
                x.copy_(h)
            want.append([o.detach().clone() for o in step()])
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in (0, 1, 0):
        with torch.no_grad():
            x.copy_(Ht if k == 0 else -Ht)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want[k]):
            assert torch.equal(a, b)


# --------------------------------------------------------------------------- the bounds-checking build
def _child():
    """Every kind of call on the bounds-checking build (a process loads one library): sync_check turns an
    index outside its buffer into LCE_ERR_BOUNDS."""
    import torch

    from chunked_lm_head_linear_gb300 import build, lce
    lce.load(build.build(checks=True))
    for N, d, V, K, chunk in [(1, 64, 37, 5, 0), (3, 72, 2, 2, 0), (33, 136, 129, 100, 0), (96, 64, 4099, 3, 0),
                              (97, 8, 257, 128, 0), (129, 136, 70001, 20, 64), (513, 256, 1000, 33, 200)]:
        rng, H, W, y = make(N, d, V, seed=N)
        idx, t = teacher(rng, N, V, K)
        Ht, Wt = heads(H, W)
        g = dev(rng.standard_normal(N).astype(np.float32))
        kept = torch.empty(N, lce.lce_logits_stride(V), device="cuda")
        for logits in (None, kept):
            kw = dict(logits=logits, chunk_tokens=chunk, sync_check=True)
            out = lce.lce_logprobs(Ht, Wt, dev(y), top_k=K, **kw)
            check_scores(out, H, W, y, 1.0, K)
            for dt in (torch.float32, torch.bfloat16):
                dH, dW = lce.lce_logprobs_backward(Ht, Wt, dev(y), out[0], out[1], out[2], g, g, dW_dtype=dt, **kw)
                check_grads(dH, dW if dt == torch.float32 else None,
                            oracle.logprobs_backward_f64(H, W, y, np64(g), np64(g)), scaled=True)
        lce.lce_logprobs(Ht, Wt, dev(y), chunk_tokens=chunk, sync_check=True)
        out = lce.lce_distill_fwd_bwd(Ht, Wt, dev(idx), dev(t), chunk_tokens=chunk, sync_check=True)
        check_grads(out[2], out[3], oracle.distill_f64(H, W, idx, t))
        lce.lce_distill_forward(Ht, Wt, dev(idx), dev(t), chunk_tokens=chunk, sync_check=True)
    print("checked build: ok")


def test_bounds_checking_build(cuda_lib):
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([os.path.dirname(here), here]))
    r = subprocess.run([sys.executable, "-c", "import test_tokens_gpu as t; t._child()"], env=env, cwd=here,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "checked build: ok" in r.stdout, (r.stdout + r.stderr)[-3000:]
