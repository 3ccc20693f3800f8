"""The losses on log-probabilities and the layer norm without a GPU: the oracle
against PyTorch's autograd, differences and closed forms; the C calls' and the
binding's refusals; the autograd modules on fakes of the calls."""
import ctypes

import numpy as np
import pytest

import oracle
from chunked_lm_head_linear_gb300 import lce

FAKE = 1 << 20   # an aligned address that is never read: refused calls stop on the host


@pytest.fixture(scope="module")
def lib():
    from chunked_lm_head_linear_gb300 import build
    build.build()
    return lce.load()


def inputs(N=12, d=16, V=29, seed=0):
    rng = np.random.default_rng(seed)
    H, W = rng.standard_normal((N, d)), rng.standard_normal((V, d)) * 0.6
    y = rng.integers(0, V, N)
    y[[1, 7]] = oracle.IGNORE_INDEX
    return rng, H, W, y


# --------------------------------------------------------------------------- the oracle
@pytest.mark.parametrize("kl", ["none", "k1", "k2", "k3"])
@pytest.mark.parametrize("dual", [0.0, 1.5])
@pytest.mark.parametrize("old", [True, False])
def test_policy_oracle_matches_autograd(kl, dual, old):
    torch = pytest.importorskip("torch")
    rng, H, W, y = inputs()
    N = len(y)
    A, w = rng.standard_normal(N), rng.random(N)
    old_logp = rng.standard_normal(N) - 3.0 if old else None
    ref = rng.standard_normal(N) - 3.0
    got = oracle.policy_f64(H, W, y, A, old_logp, ref, w, temperature=0.8, kl=kl, kl_coef=0.3, dual_clip=dual,
                            clip_high=0.3, grad_loss=1.7)
    h, ww = torch.tensor(H, requires_grad=True), torch.tensor(W, requires_grad=True)
    told = torch.tensor(y) >= 0
    logq = torch.log_softmax(h @ ww.t() / 0.8, 1)
    logp = logq[told, torch.tensor(y)[told]]
    a = torch.tensor(A)[told]
    r = torch.exp(logp - (torch.tensor(old_logp)[told] if old else logp.detach()))
    # torch splits the gradient where both sides are equal; the parts add up inside the range
    s = torch.minimum(r * a, r.clamp(0.8, 1.3) * a)
    if dual:
        s = torch.where(a < 0, torch.maximum(s, dual * a), s)
    row = -s
    u = logp - torch.tensor(ref)[told]
    if kl != "none":
        row = row + 0.3 * {"k1": u, "k2": u * u / 2, "k3": torch.exp(-u) - 1 + u}[kl]
    loss = (row * torch.tensor(w)[told]).sum() / told.sum()
    dH, dW = torch.autograd.grad(1.7 * loss, [h, ww])
    assert abs(loss.item() - got["loss"]) < 1e-13
    np.testing.assert_allclose(got["dH"], dH.numpy(), rtol=1e-10, atol=1e-13)
    np.testing.assert_allclose(got["dW"], dW.numpy(), rtol=1e-10, atol=1e-13)
    assert (got["row_loss"][[1, 7]] == 0).all() and (got["logp"][[1, 7]] == 0).all()


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
@pytest.mark.parametrize("average", [True, False])
def test_preference_oracle_matches_autograd(kind, average):
    torch = pytest.importorskip("torch")
    rng, H, W, y = inputs(N=20)
    cu = np.array([1, 5, 9, 9, 14, 16, 18])   # an empty sequence, rows before and behind
    ref = rng.standard_normal(6)
    kw = dict(kind=kind, beta=0.4, label_smoothing=0.1 if kind == "sigmoid" else 0.0, margin=0.0 if kind == "ipo" else 0.2)
    got = oracle.preference_f64(H, W, y, cu, ref, average=average, grad_loss=0.6, **kw)
    h, w = torch.tensor(H, requires_grad=True), torch.tensor(W, requires_grad=True)
    logq = torch.log_softmax(h @ w.t(), 1)
    S = []
    for s in range(6):
        rows = [i for i in range(cu[s], cu[s + 1]) if y[i] >= 0]
        part = sum((logq[i, y[i]] for i in rows), torch.zeros((), dtype=torch.float64))
        S.append(part / max(len(rows), 1) if average else part)
    S = torch.stack(S)
    ratio = S - torch.tensor(ref)
    delta = ratio[0::2] - ratio[1::2]
    x = 0.4 * delta - kw["margin"]
    ls = torch.nn.functional.logsigmoid
    pair = {"sigmoid": -0.9 * ls(x) - 0.1 * ls(-x), "hinge": torch.relu(1 - x), "ipo": (delta - 1 / 0.8) ** 2}[kind]
    dH, dW = torch.autograd.grad(0.6 * pair.mean(), [h, w])
    np.testing.assert_allclose(got["pair_loss"], pair.detach().numpy(), rtol=1e-12)
    np.testing.assert_allclose(got["seq_logp"], S.detach().numpy(), rtol=1e-12)
    np.testing.assert_allclose(got["dH"], dH.numpy(), rtol=1e-9, atol=1e-14)
    np.testing.assert_allclose(got["dW"], dW.numpy(), rtol=1e-9, atol=1e-14)
    assert not got["dH"][[0, 18, 19]].any()


def test_oracle_gradients_match_differences():
    rng, H, W, y = inputs(N=8, d=6, V=9)
    A, old, ref = rng.standard_normal(8), rng.standard_normal(8) - 2.0, rng.standard_normal(8) - 2.0
    cu = np.array([0, 2, 4, 7, 8])
    x, w, dH = rng.standard_normal((5, 16)), rng.standard_normal(16), rng.standard_normal((5, 16))
    losses = {
        "policy": (lambda h, v: oracle.policy_f64(h, v, y, A, old, ref, kl="k3", kl_coef=0.5)["loss"],
                   oracle.policy_f64(H, W, y, A, old, ref, kl="k3", kl_coef=0.5)),
        "preference": (lambda h, v: oracle.preference_f64(h, v, y, cu, beta=0.7)["loss"],
                       oracle.preference_f64(H, W, y, cu, beta=0.7)),
    }
    e = 1e-6
    for name, (f, got) in losses.items():
        for k, M in (("dH", H), ("dW", W)):
            for i, j in [(0, 0), (2, 3), (5, 1), (6, 4)]:
                D = np.zeros_like(M)
                D[i, j] = e
                up, down = (f(H + D, W), f(H - D, W)) if k == "dH" else (f(H, W + D), f(H, W - D))
                assert abs((up - down) / (2 * e) - got[k][i, j]) < 1e-8, (name, k, i, j)
    got = oracle.layernorm_backward_f64(x, w, dH)
    F = lambda a, b: (oracle.layernorm_f64(a, b, None)["H"] * dH).sum()  # noqa: E731
    for i, j in [(0, 0), (3, 9)]:
        D = np.zeros_like(x)
        D[i, j] = e
        assert abs((F(x + D, w) - F(x - D, w)) / (2 * e) - got["dx"][i, j]) < 1e-7
        d = np.zeros_like(w)
        d[j] = e
        assert abs((F(x, w + d) - F(x, w - d)) / (2 * e) - got["dw"][j]) < 1e-7


def test_oracle_closed_forms():
    one = np.ones(3, bool)
    logp = np.log(np.array([0.5, 0.25, 0.125]))
    # ratios 2, 1, 0.5: clipped from above, free, and (negative advantage) clipped from below
    row, a = oracle.policy_rows_f64(logp, one, np.array([1.0, 1.0, -1.0]), np.log(np.array([0.25, 0.25, 0.25])))
    np.testing.assert_allclose(row, [-1.2, -1.0, 0.8])
    np.testing.assert_allclose(a, [0.0, -1.0, 0.0])
    # a ratio of 8 against a negative advantage, bounded by the dual clip
    row, a = oracle.policy_rows_f64(np.zeros(1), one[:1], np.array([-1.0]), np.log(np.array([0.125])), dual_clip=3.0)
    assert row[0] == 3.0 and a[0] == 0.0
    for kl in ("k1", "k2", "k3"):   # no divergence, no share of the term
        row, a = oracle.policy_rows_f64(logp, one, np.zeros(3), None, logp, kl=kl, kl_coef=2.0)
        assert not row.any() and (kl == "k1" or not a.any())
    loss, slope = oracle.preference_pairs_f64(np.array([-3.0, -3.0]))
    assert abs(loss[0] - np.log(2)) < 1e-15 and abs(slope[0] + 0.05) < 1e-15
    f = oracle.layernorm_f64(np.full((1, 8), 3.0), np.arange(8.0), np.ones(8))
    assert (f["H"] == 1.0).all() and f["mean"][0] == 3.0


# --------------------------------------------------------------------------- refusals
def policy(**kw):
    p = dict(clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0, kl=0, reserved=0)
    p.update(kw)
    return lce.LcePolicy(*p.values())


def preference(**kw):
    p = dict(beta=0.1, label_smoothing=0.0, margin=0.0, kind=0, flags=0, reserved=0)
    p.update(kw)
    return lce.LcePreference(*p.values())


def test_policy_refusals(lib):
    E, P, nan, inf = lce, FAKE, float("nan"), float("inf")

    def call(grad=True, H=P, W=P, y=P, N=64, d=64, V=1000, T=1.0, pol=None, adv=P, old=P, ref=P, w=P, g=None, grads=0,
             loss=P, logp=P, row=P, dH=P, dW=P, opts=None, ws=P, nbytes=1 << 40):
        o = opts if opts is not None else lce.make_opts()
        pol = policy() if pol is None else pol
        pol = None if pol == "null" else ctypes.byref(pol)
        if grad:
            return lib.lce_policy_fwd_bwd(H, W, y, N, d, V, T, pol, adv, old, ref, w, g, grads, loss, logp, row, dH, dW,
                                          ctypes.byref(o), ws, nbytes, None)
        return lib.lce_policy_forward(H, W, y, N, d, V, T, pol, adv, old, ref, w, loss, logp, row, ctypes.byref(o), ws,
                                      nbytes, None)

    for grad in (True, False):
        for bad in (dict(H=None), dict(W=None), dict(y=None), dict(adv=None), dict(loss=None), dict(logp=None),
                    dict(row=None), dict(ws=None), dict(pol="null"), dict(N=-1), dict(d=12), dict(V=0), dict(T=0.0),
                    dict(V=2 ** 31 - 1), dict(pol=policy(clip_low=-0.1)), dict(pol=policy(clip_low=nan)),
                    dict(pol=policy(clip_high=nan)), dict(pol=policy(clip_high=-1.0)), dict(pol=policy(dual_clip=0.5)),
                    dict(pol=policy(dual_clip=nan)), dict(pol=policy(kl_coef=inf)), dict(pol=policy(kl_coef=nan)),
                    dict(pol=policy(kl=4)), dict(pol=policy(kl=-1)), dict(pol=policy(reserved=1)),
                    dict(pol=policy(kl=3), ref=None), dict(opts=lce.make_opts(reserved=E.LCE_TEST_FORCE_TIMEOUT)),
                    dict(opts=lce.make_opts(reduction=3))):
            assert call(grad, **bad) == E.LCE_ERR_INVALID_ARG, (grad, bad)
        for bad in (dict(H=P + 8), dict(W=P + 2), dict(y=P + 4), dict(adv=P + 2), dict(old=P + 1), dict(ref=P + 2),
                    dict(w=P + 2), dict(loss=P + 1), dict(logp=P + 2), dict(row=P + 2), dict(ws=P + 128)):
            assert call(grad, **bad) == E.LCE_ERR_ALIGNMENT, (grad, bad)
        need = lce.lce_policy_workspace_size(64, 64, 1000, grad)
        assert call(grad, nbytes=need - 1) == E.LCE_ERR_WORKSPACE
    for bad in (dict(dH=None, dW=None), dict(grads=2), dict(grads=1, opts=lce.make_opts(accumulate_dW=True))):
        assert call(**bad) == E.LCE_ERR_INVALID_ARG, bad
    for bad in (dict(dH=P + 8), dict(dW=P + 4), dict(g=P + 2)):
        assert call(**bad) == E.LCE_ERR_ALIGNMENT, bad
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():   # these get as far as the device check
        for good in (dict(), dict(old=None), dict(ref=None), dict(w=None), dict(dH=None), dict(dW=None), dict(grads=1),
                     dict(grad=False), dict(pol=policy(kl=3, kl_coef=-1.0)), dict(pol=policy(clip_high=inf)),
                     dict(pol=policy(clip_low=2.0, dual_clip=1.0)),
                     dict(N=0, H=None, y=None, adv=None, old=None, ref=None, w=None, logp=None, row=None, dH=None)):
            assert call(**good) in (E.LCE_ERR_CUDA, E.LCE_ERR_UNSUPPORTED_DEVICE), good


def test_preference_refusals(lib):
    E, P, nan, inf = lce, FAKE, float("nan"), float("inf")

    def call(grad=True, H=P, W=P, y=P, N=64, d=64, V=1000, cu=P, pairs=3, T=1.0, pref=None, ref=P, g=None, grads=0,
             loss=P, pl=P, sl=P, dH=P, dW=P, opts=None, ws=P, nbytes=1 << 40):
        o = opts if opts is not None else lce.make_opts()
        pref = preference() if pref is None else pref
        pref = None if pref == "null" else ctypes.byref(pref)
        if grad:
            return lib.lce_preference_fwd_bwd(H, W, y, N, d, V, cu, pairs, T, pref, ref, g, grads, loss, pl, sl, dH, dW,
                                              ctypes.byref(o), ws, nbytes, None)
        return lib.lce_preference_forward(H, W, y, N, d, V, cu, pairs, T, pref, ref, loss, pl, sl, ctypes.byref(o), ws,
                                          nbytes, None)

    for grad in (True, False):
        for bad in (dict(H=None), dict(W=None), dict(y=None), dict(cu=None), dict(loss=None), dict(pl=None),
                    dict(sl=None), dict(ws=None), dict(pref="null"), dict(N=-1), dict(d=4), dict(V=0), dict(T=nan),
                    dict(pairs=-1), dict(pairs=1 << 30), dict(pref=preference(beta=0.0)), dict(pref=preference(beta=inf)),
                    dict(pref=preference(beta=nan)), dict(pref=preference(label_smoothing=0.5)),
                    dict(pref=preference(label_smoothing=-0.1)), dict(pref=preference(margin=nan)),
                    dict(pref=preference(kind=3)), dict(pref=preference(kind=-1)), dict(pref=preference(flags=4)),
                    dict(pref=preference(reserved=1)), dict(pref=preference(kind=1, label_smoothing=0.1)),
                    dict(pref=preference(kind=2, margin=0.1)), dict(opts=lce.make_opts(reserved=1))):
            assert call(grad, **bad) == E.LCE_ERR_INVALID_ARG, (grad, bad)
        for bad in (dict(H=P + 8), dict(W=P + 2), dict(y=P + 4), dict(cu=P + 4), dict(ref=P + 2), dict(loss=P + 1),
                    dict(pl=P + 2), dict(sl=P + 2), dict(ws=P + 128), dict(cu=P + 2, pref=preference(flags=2))):
            assert call(grad, **bad) == E.LCE_ERR_ALIGNMENT, (grad, bad)
        need = lce.lce_preference_workspace_size(64, 64, 1000, 3, grad)
        assert call(grad, nbytes=need - 1) == E.LCE_ERR_WORKSPACE
    for bad in (dict(dH=None, dW=None), dict(grads=2), dict(grads=1, opts=lce.make_opts(accumulate_dW=True))):
        assert call(**bad) == E.LCE_ERR_INVALID_ARG, bad
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        for good in (dict(), dict(ref=None), dict(dH=None), dict(dW=None), dict(grads=1), dict(grad=False),
                     dict(cu=P + 4, pref=preference(flags=3)), dict(pairs=0, cu=None, pl=None, sl=None),
                     dict(N=0, H=None, y=None, dH=None), dict(pref=preference(kind=1, margin=-2.0)),
                     dict(pref=preference(kind=2))):
            assert call(**good) in (E.LCE_ERR_CUDA, E.LCE_ERR_UNSUPPORTED_DEVICE), good


def test_layernorm_refusals(lib):
    E, P, nan = lce, FAKE, float("nan")

    def fwd(x=P, w=P, b=P, N=4, d=64, eps=1e-5, types=0, H=P, mean=P, rstd=P):
        return lib.lce_layernorm_forward(x, w, b, N, d, eps, types, H, mean, rstd, None)

    def bwd(x=P, w=P, mean=P, rstd=P, dH=P, N=4, d=64, types=0, dx=P, dw=P, db=P, ws=P, nbytes=1 << 40):
        return lib.lce_layernorm_backward(x, w, mean, rstd, dH, N, d, types, dx, dw, db, ws, nbytes, None)

    for bad in (dict(x=None), dict(H=None), dict(N=-1), dict(d=12), dict(d=0), dict(d=32776), dict(eps=-1.0),
                dict(eps=nan), dict(eps=float("inf")), dict(types=4), dict(types=-1)):
        assert fwd(**bad) == E.LCE_ERR_INVALID_ARG, bad
    for bad in (dict(x=P + 8), dict(w=P + 4), dict(b=P + 8), dict(H=P + 2), dict(mean=P + 2), dict(rstd=P + 1)):
        assert fwd(**bad) == E.LCE_ERR_ALIGNMENT, bad
    for bad in (dict(x=None), dict(mean=None), dict(rstd=None), dict(dH=None), dict(dx=None, dw=None, db=None),
                dict(ws=None), dict(N=-1), dict(d=20), dict(types=8)):
        assert bwd(**bad) == E.LCE_ERR_INVALID_ARG, bad
    for bad in (dict(x=P + 8), dict(w=P + 4), dict(dH=P + 8), dict(dx=P + 2), dict(dw=P + 2), dict(db=P + 2),
                dict(mean=P + 2), dict(rstd=P + 2), dict(ws=P + 64)):
        assert bwd(**bad) == E.LCE_ERR_ALIGNMENT, bad
    assert bwd(nbytes=lce.lce_layernorm_workspace_size(4, 64) - 1) == E.LCE_ERR_WORKSPACE
    assert lce.lce_layernorm_workspace_size(4, 12) == 0 and lce.lce_layernorm_workspace_size(-1, 8) == 0
    assert lce.lce_layernorm_workspace_size(0, 8) > 0
    assert lce.lce_layernorm_workspace_size(1 << 20, 4096) < 64 << 20   # does not grow with N without end
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        for rc in (fwd(), fwd(w=None, b=None), fwd(mean=None, rstd=None), fwd(types=3), fwd(eps=0.0), fwd(N=0, x=None, H=None),
                   bwd(), bwd(dx=None), bwd(w=None, dw=None, db=None, ws=None, nbytes=0), bwd(d=32768), bwd(db=None),
                   bwd(N=0, x=None, mean=None, rstd=None, dH=None, dx=None)):
            assert rc in (E.LCE_ERR_CUDA, E.LCE_ERR_UNSUPPORTED_DEVICE)


def test_workspaces_grow_with_the_chunk_only(lib):
    o = lce.make_opts(chunk_tokens=1024)
    V, d = 151936, 2048
    for grad in (True, False):   # a few floats a row more
        for size in (lambda n: lce.lce_policy_workspace_size(n, d, V, grad, 0, o),
                     lambda n: lce.lce_preference_workspace_size(n, d, V, 4, grad, 0, o)):
            assert 0 <= size(65536) - size(8192) <= (65536 - 8192) * 16
    assert lce.lce_policy_workspace_size(64, 7, V) == 0 and lce.lce_preference_workspace_size(64, 8, V, -1) == 0
    # a bf16 dW over several chunks is summed in fp32
    assert lce.lce_policy_workspace_size(8192, d, V, True, 1, o) - lce.lce_policy_workspace_size(8192, d, V, True, 0, o) >= 4 * V * d


def test_binding_refuses_what_does_not_fit():
    torch = pytest.importorskip("torch")
    H, W = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(3, 8, dtype=torch.bfloat16)
    y, f, cu = torch.zeros(4, dtype=torch.int64), torch.zeros(4), torch.tensor([0, 2, 4])
    for call in (lambda: lce.lce_policy_forward(H, W, y, f), lambda: lce.lce_policy_fwd_bwd(H, W, y, f),
                 lambda: lce.lce_preference_forward(H, W, y, cu), lambda: lce.lce_preference_fwd_bwd(H, W, y, cu),
                 lambda: lce.lce_layernorm_forward(f.view(1, 4)),
                 lambda: lce.lce_layernorm_backward(f.view(1, 4), None, f, f, H)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


# --------------------------------------------------------------------------- the autograd modules, on fakes of the calls
def test_modules_on_fakes(monkeypatch):
    """What the modules call, with grad mode and without, with a frozen side, and what their backward hands out."""
    torch = pytest.importorskip("torch")
    from chunked_lm_head_linear_gb300.autograd import FusedLayerNorm, FusedLinearPolicyLoss, FusedLinearPreferenceLoss
    seen = []

    def fwd(name, n):
        def call(H, W, y, *a, **kw):
            seen.append(name)
            return torch.zeros(1), torch.zeros(n), torch.zeros(n)
        return call

    def both(name, n):
        def call(H, W, y, *a, need_dH, need_dW, dW_dtype, **kw):
            seen.append((name, need_dH, need_dW))
            assert dW_dtype == W.dtype
            return (torch.zeros(1), torch.zeros(n), torch.zeros(n), torch.ones_like(H) if need_dH else None,
                    torch.ones_like(W) if need_dW else None)
        return call

    def scale(dH, dW, g):
        for t in (dH, dW):
            if t is not None:
                t.mul_(g.to(t.dtype))

    for name, n in (("policy", 4), ("preference", 4)):
        monkeypatch.setattr(lce, f"lce_{name}_forward", fwd(name, n))
        monkeypatch.setattr(lce, f"lce_{name}_fwd_bwd", both(name, n))
    monkeypatch.setattr(lce, "lce_scale_grads_bfloat", scale)
    H, W = torch.zeros(4, 8).bfloat16(), torch.zeros(3, 8).bfloat16()
    y, f, cu = torch.zeros(4, dtype=torch.int64), torch.zeros(4), torch.tensor([0, 1, 2, 3, 4])
    for name, module, args in (("policy", FusedLinearPolicyLoss(), (y, f)),
                               ("preference", FusedLinearPreferenceLoss(), (y, cu))):
        seen.clear()
        with torch.no_grad():
            module(H.requires_grad_(True), W.requires_grad_(True), *args)
        module(H.detach(), W.detach(), *args)
        assert seen == [name, name]
        for a, b in ((True, True), (True, False), (False, True)):
            h, w = H.detach().requires_grad_(a), W.detach().requires_grad_(b)
            seen.clear()
            loss, extra = module(h, w, *args)
            assert seen == [(name, a, b)] and loss.shape == () and not extra.requires_grad
            loss.mul(2.0).backward(retain_graph=True)
            for t, need in ((h, a), (w, b)):
                assert (t.grad == 2.0).all() if need else t.grad is None
            with pytest.raises(RuntimeError, match="run the forward again"):
                loss.backward()
    monkeypatch.setattr(lce, "lce_layernorm_forward", lambda x, w, b, eps: (x.bfloat16(), torch.zeros(4), torch.ones(4)))

    def ln_bwd(x, w, mean, rstd, dH, *, bias, need_dx, need_dw):
        seen.append((need_dx, need_dw, bias))
        return (torch.ones_like(x) if need_dx else None, torch.ones(8) if need_dw else None,
                torch.ones(8) if bias else None)

    monkeypatch.setattr(lce, "lce_layernorm_backward", ln_bwd)
    seen.clear()
    x, w, b = torch.zeros(4, 8, requires_grad=True), torch.ones(8).bfloat16().requires_grad_(True), torch.zeros(8).bfloat16()
    FusedLayerNorm()(x, w, b).sum().backward()
    assert seen == [(True, True, False)] and x.grad.dtype == torch.float32 and w.grad.dtype == torch.bfloat16
