"""The head's token operators without a GPU: the fp64 oracle pinned against
PyTorch's autograd, differences and closed forms, and the refusals of the C
calls and the binding."""
import ctypes

import numpy as np
import pytest

import oracle
from chunked_lm_head_linear_gb300 import build, lce

FAKE = 0x100000  # an aligned non-null address; never dereferenced by host-side checks


@pytest.fixture(scope="module")
def lib():
    build.build()
    return lce.load()


def _case(N=7, d=8, V=23, seed=0):
    rng = np.random.default_rng(seed)
    H, W = rng.standard_normal((N, d)), 0.5 * rng.standard_normal((V, d))
    y = rng.integers(0, V, N)
    y[1] = oracle.IGNORE_INDEX
    return rng, H, W, y


# --------------------------------------------------------------------------- oracle
@pytest.mark.parametrize("T", [1.0, 0.6, 2.5])
def test_logprobs_oracle_matches_autograd(T):
    torch = pytest.importorskip("torch")
    rng, H, W, y = _case()
    g1, g2 = rng.standard_normal(len(H)), rng.standard_normal(len(H))
    Ht, Wt = torch.tensor(H, requires_grad=True), torch.tensor(W, requires_grad=True)
    logq = torch.log_softmax(Ht @ Wt.T / T, 1)
    yt = torch.tensor(y)
    logp = torch.where(yt >= 0, logq.gather(1, yt.clamp(min=0)[:, None])[:, 0], 0.0)
    ent = -(logq.exp() * logq).sum(1)
    (logp @ torch.tensor(g1) + ent @ torch.tensor(g2)).backward()
    f = oracle.logprobs_f64(H, W, y, temperature=T, top_k=5)
    b = oracle.logprobs_backward_f64(H, W, y, g1, g2, temperature=T)
    for a, ref in ((f["logp"], logp), (f["entropy"], ent), (f["lse"], torch.logsumexp(Ht @ Wt.T / T, 1)),
                   (f["top_logp"], logq.topk(5, 1).values), (b["dH"], Ht.grad), (b["dW"], Wt.grad)):
        np.testing.assert_allclose(a, ref.detach().numpy(), rtol=1e-12, atol=1e-13)
    assert (f["top_idx"] == logq.topk(5, 1).indices.numpy()).all()


@pytest.mark.parametrize("T,renormalize", [(1.0, True), (2.0, True), (1.0, False)])
def test_distill_oracle_matches_autograd(T, renormalize):
    torch = pytest.importorskip("torch")
    rng, H, W, _ = _case()
    N, V, K = len(H), len(W), 4
    idx = np.stack([rng.permutation(V)[:K] for _ in range(N)])
    t = 2 * rng.standard_normal((N, K))
    if not renormalize:
        t -= 4.0
    idx[2, 2:] = oracle.IGNORE_INDEX   # a shorter list
    idx[3] = oracle.IGNORE_INDEX       # no list
    t[4, 1] = -np.inf
    idx[5, 1] = idx[5, 0]              # the same token twice
    Ht, Wt = torch.tensor(H, requires_grad=True), torch.tensor(W, requires_grad=True)
    logq = torch.log_softmax(Ht @ Wt.T / T, 1)
    it, tt = torch.tensor(idx), torch.tensor(t)
    kept = (it >= 0) & (tt > -np.inf)
    q = torch.where(kept, (tt / T).exp(), 0.0)
    if renormalize:
        q = q / q.sum(1, keepdim=True).clamp(min=1e-300)
    loss = T * T * (torch.special.xlogy(q, q) - q * logq.gather(1, it.clamp(min=0))).sum() / 6
    (3.0 * loss).backward()
    r = oracle.distill_f64(H, W, idx, t, temperature=T, renormalize=renormalize, grad_loss=3.0)
    np.testing.assert_allclose(r["loss"], loss.item(), rtol=1e-12)
    np.testing.assert_allclose(r["dH"], Ht.grad.numpy(), rtol=1e-11, atol=1e-14)
    np.testing.assert_allclose(r["dW"], Wt.grad.numpy(), rtol=1e-11, atol=1e-14)
    assert r["row_loss"][3] == 0 and not r["dH"][3].any()


def test_oracle_gradients_match_differences():
    """Central differences, h = 1e-5: truncation h^2 f'''/6 and rounding 2e-16 |f| / h stay below 1e-9."""
    rng, H, W, y = _case(N=4, d=4, V=9)
    g1, g2 = rng.standard_normal(4), rng.standard_normal(4)
    idx = np.stack([rng.permutation(9)[:3] for _ in range(4)])
    t = rng.standard_normal((4, 3))

    def f_logp(H, W):
        r = oracle.logprobs_f64(H, W, y, temperature=0.8)
        return r["logp"] @ g1 + r["entropy"] @ g2

    def f_kd(H, W):
        return oracle.distill_f64(H, W, idx, t, temperature=1.7)["loss"]

    for f, b in ((f_logp, oracle.logprobs_backward_f64(H, W, y, g1, g2, temperature=0.8)),
                 (f_kd, oracle.distill_f64(H, W, idx, t, temperature=1.7))):
        for _ in range(5):
            U, S = rng.standard_normal(H.shape), rng.standard_normal(W.shape)
            h = 1e-5
            diff = (f(H + h * U, W + h * S) - f(H - h * U, W - h * S)) / (2 * h)
            assert abs(diff - (b["dH"] * U).sum() - (b["dW"] * S).sum()) < 1e-7


def test_oracle_closed_forms():
    y = np.array([2, oracle.IGNORE_INDEX])
    r = oracle.logprobs_f64(np.zeros((2, 4)), np.ones((6, 4)), y, top_k=3)
    np.testing.assert_allclose(r["logp"], [-np.log(6), 0])
    np.testing.assert_allclose(r["entropy"], np.log(6))
    assert (r["top_idx"] == [0, 1, 2]).all()           # all equal: the lowest indices
    # a teacher equal to the student: no loss, no gradient
    rng, H, W, _ = _case(N=3, V=5)
    z = H @ W.T
    idx = np.tile(np.arange(5), (3, 1))
    r = oracle.distill_f64(H, W, idx, z, temperature=3.0)
    assert abs(r["loss"]) < 1e-14 and np.abs(r["dH"]).max() < 1e-15


# --------------------------------------------------------------------------- refusals
def test_logprobs_refusals(lib):
    E, P = lce, FAKE

    def call(H=P, W=P, y=P, N=64, d=64, V=1000, T=1.0, K=5, logp=P, lse=P, ent=P, tl=P, ti=P, kept=None, opts=None,
             ws=P, nbytes=1 << 40):
        o = opts if opts is not None else lce.make_opts()
        return lib.lce_logprobs(H, W, y, N, d, V, T, K, logp, lse, ent, tl, ti, kept, ctypes.byref(o), ws, nbytes,
                                None)

    for bad in (dict(H=None), dict(W=None), dict(y=None), dict(logp=None), dict(lse=None), dict(tl=None),
                dict(ti=None), dict(ws=None), dict(N=-1), dict(d=12), dict(V=0), dict(T=0.0), dict(T=-1.0),
                dict(T=float("nan")), dict(T=float("inf")), dict(T=9e-7), dict(T=2e6), dict(V=2 ** 31 - 1), dict(V=2 ** 31 - 65535), dict(K=-1), dict(K=E.LCE_MAX_TOP + 1), dict(K=6, V=5),
                dict(opts=lce.make_opts(reserved=1)), dict(opts=lce.make_opts(chunk_tokens=-1))):
        assert call(**bad) == E.LCE_ERR_INVALID_ARG, bad
    for bad in (dict(H=P + 8), dict(W=P + 2), dict(y=P + 4), dict(logp=P + 1), dict(lse=P + 2), dict(ent=P + 2),
                dict(tl=P + 2), dict(ti=P + 4), dict(ws=P + 128), dict(kept=P + 8)):
        assert call(**bad) == E.LCE_ERR_ALIGNMENT, bad
    need = lce.lce_logprobs_workspace_size(64, 64, 1000, 5)
    assert call(nbytes=need - 1) == E.LCE_ERR_WORKSPACE
    less = lce.lce_logprobs_workspace_size(64, 64, 1000, 0)   # enough when the caller keeps the logits
    assert less < need and call(kept=P, nbytes=less - 1) == E.LCE_ERR_WORKSPACE
    assert [lce.lce_logits_stride(v) for v in (1, 256, 257, 151655)] == [256, 256, 512, 151808]
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():   # these get as far as the device check
        for good in (dict(), dict(ent=None), dict(K=0, tl=None, ti=None), dict(nbytes=need), dict(V=2 ** 31 - 65536, nbytes=1 << 50),
                     dict(kept=P, nbytes=less),
                     dict(N=0, H=None, y=None, logp=None, lse=None, tl=None, ti=None)):
            assert call(**good) in (E.LCE_ERR_CUDA, E.LCE_ERR_UNSUPPORTED_DEVICE), good


def test_logprobs_backward_refusals(lib):
    E, P = lce, FAKE

    def call(logp=P, lse=P, ent=P, g1=P, g2=P, kept=None, grads=0, dH=P, dW=P, T=1.0, N=64, acc=False,
             reserved=0, nbytes=1 << 40):
        o = lce.make_opts(accumulate_dW=acc, chunk_tokens=32, reserved=reserved)
        return lib.lce_logprobs_backward(P, P, P, N, 64, 1000, T, logp, lse, ent, g1, g2, kept, grads, dH, dW,
                                         ctypes.byref(o), P, nbytes, None)

    for bad in (dict(logp=None), dict(lse=None), dict(g1=None), dict(ent=None), dict(dH=None, dW=None), dict(T=0.0), dict(N=-2),
                dict(grads=2), dict(grads=E.LCE_DW_BF16, acc=True), dict(reserved=E.LCE_TEST_FORCE_TIMEOUT)):
        assert call(**bad) == E.LCE_ERR_INVALID_ARG, bad
    for bad in (dict(kept=P + 4), dict(logp=P + 1), dict(lse=P + 2), dict(ent=P + 2), dict(g1=P + 2), dict(g2=P + 1), dict(dH=P + 8), dict(dW=P + 4)):
        assert call(**bad) == E.LCE_ERR_ALIGNMENT, bad
    o = lce.make_opts(chunk_tokens=32)
    sizes = [lce.lce_logprobs_backward_workspace_size(64, 64, 1000, g, o) for g in (0, E.LCE_DW_BF16)]
    assert sizes[1] - sizes[0] >= 1000 * 64 * 4       # two chunks: the fp32 sum of a bf16 dW
    one = [lce.lce_logprobs_backward_workspace_size(64, 64, 1000, g) for g in (0, E.LCE_DW_BF16)]
    assert one[0] == one[1] and lce.lce_logprobs_backward_workspace_size(64, 64, 1000, 4) == 0
    for g in (0, 1):
        assert call(grads=g, nbytes=sizes[g] - 1) == E.LCE_ERR_WORKSPACE
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        for good in (dict(), dict(ent=None, g2=None), dict(dH=None), dict(dW=None), dict(N=0), dict(kept=P), dict(grads=1)):
            assert call(**good) in (E.LCE_ERR_CUDA, E.LCE_ERR_UNSUPPORTED_DEVICE), good


def test_distill_refusals(lib):
    E, P = lce, FAKE

    def call(grad=True, H=P, W=P, idx=P, t=P, N=64, d=64, V=1000, K=5, teacher=0, T=1.0, loss=P, row=P, dH=P, dW=P,
             grads=0, opts=None, nbytes=1 << 40):
        o = opts if opts is not None else lce.make_opts()
        if grad:
            return lib.lce_distill_fwd_bwd(H, W, idx, t, N, d, V, K, teacher, T, None, grads, loss, row, dH, dW,
                                           ctypes.byref(o), P, nbytes, None)
        return lib.lce_distill_forward(H, W, idx, t, N, d, V, K, teacher, T, loss, row, ctypes.byref(o), P, nbytes,
                                       None)

    for grad in (True, False):
        for bad in (dict(H=None), dict(W=None), dict(idx=None), dict(t=None), dict(loss=None), dict(row=None),
                    dict(K=0), dict(K=E.LCE_MAX_TOP + 1), dict(teacher=4), dict(teacher=-1), dict(T=0.0),
                    dict(T=2.0, teacher=E.LCE_TEACHER_LOGPROBS), dict(V=-1), dict(d=4),
                    dict(opts=lce.make_opts(reduction=3))):
            assert call(grad, **bad) == E.LCE_ERR_INVALID_ARG, (grad, bad)
        for bad in (dict(H=P + 8), dict(idx=P + 4), dict(t=P + 2), dict(t=P + 1, teacher=1), dict(row=P + 2)):
            assert call(grad, **bad) == E.LCE_ERR_ALIGNMENT, (grad, bad)
        need = lce.lce_distill_workspace_size(64, 64, 1000, 5, grad)
        assert call(grad, nbytes=need - 1) == E.LCE_ERR_WORKSPACE
    for bad in (dict(dH=None, dW=None), dict(grads=8), dict(grads=1, opts=lce.make_opts(accumulate_dW=True))):
        assert call(**bad) == E.LCE_ERR_INVALID_ARG, bad
    assert call(dW=P + 4) == E.LCE_ERR_ALIGNMENT
    assert lce.lce_distill_workspace_size(64, 64, 1000, 5, True) > lce.lce_distill_workspace_size(64, 64, 1000, 5, False)
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        for good in (dict(), dict(dH=None), dict(dW=None), dict(grad=False), dict(t=P + 2, teacher=1), dict(grads=1),
                     dict(teacher=E.LCE_TEACHER_LOGPROBS)):
            assert call(**good) in (E.LCE_ERR_CUDA, E.LCE_ERR_UNSUPPORTED_DEVICE), good


def test_token_workspaces_grow_with_the_chunk_only():
    o = lce.make_opts(chunk_tokens=1024)
    V, d = 151936, 2048
    for size in (lambda n: lce.lce_logprobs_workspace_size(n, d, V, 20, o),
                 lambda n: lce.lce_logprobs_backward_workspace_size(n, d, V, 0, o),
                 lambda n: lce.lce_distill_workspace_size(n, d, V, 64, True, 0, o)):
        assert size(65536) == size(8192) > 0
    assert lce.lce_logprobs_workspace_size(8192, d, V, 0, o) < lce.lce_logprobs_workspace_size(8192, d, V, 1, o)
    assert lce.lce_logprobs_workspace_size(64, 7, V, 0) == 0 and lce.lce_logprobs_workspace_size(64, 8, 4, 5) == 0
    assert lce.lce_distill_workspace_size(64, 8, V, 0) == 0 and lce.lce_distill_workspace_size(64, 8, V, 129) == 0


def test_scale_refusals(lib):
    E, P = lce, FAKE
    call = lib.lce_scale_grads_bfloat
    assert call(P, P, 4, 12, 4, P, None) == E.LCE_ERR_INVALID_ARG
    assert call(P, P, 4, 8, 4, None, None) == E.LCE_ERR_INVALID_ARG
    assert call(P + 8, P, 4, 8, 4, P, None) == E.LCE_ERR_ALIGNMENT
    assert call(P, P + 2, 4, 8, 4, P, None) == E.LCE_ERR_ALIGNMENT


def test_binding_refuses_cpu_tensors_and_bad_modes():
    torch = pytest.importorskip("torch")
    H, W = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(3, 8, dtype=torch.bfloat16)
    y, f = torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    idx, t = torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2)
    for call in (lambda: lce.lce_logprobs(H, W, y), lambda: lce.lce_logprobs_backward(H, W, y, f, f, f, f),
                 lambda: lce.lce_distill_forward(H, W, idx, t), lambda: lce.lce_distill_fwd_bwd(H, W, idx, t)):
        with pytest.raises(ValueError, match="CUDA tensors"):
            call()
    with pytest.raises(ValueError, match="temperature must be 1"):
        lce._distill_mode(0, False, 2.0)
    with pytest.raises(ValueError, match="dW_dtype"):
        lce._dW_mode(torch.float16)


def test_token_chunks_are_equal_by_default():
    """chunk_tokens = 0: the workspace of equal chunks of about 4096 tokens in whole tiles, one chunk below 6144."""
    size = lambda n, c: lce.lce_logprobs_workspace_size(n, 64, 1000, 1, lce.make_opts(chunk_tokens=c))  # noqa: E731
    for n, chunk in ((1, 1), (300, 300), (4096, 4096), (5000, 5000), (6143, 6143), (7000, 3584), (8192, 4096),
                     (10000, 5120), (100000, 4352)):
        assert size(n, 0) == size(n, chunk), n


def test_kept_statistics_refusals(lib):
    """lce_logprobs_keep and lce_logprobs_keep_backward check what their plain forms check, and their stats."""
    E, P = lce, FAKE

    def fwd(stats=P, lse=P, kept=None, N=64, nbytes=1 << 40):
        o = lce.make_opts()
        return lib.lce_logprobs_keep(P, P, P, N, 64, 1000, 1.0, 0, P, lse, P, None, None, kept, stats, ctypes.byref(o), P,
                                     nbytes, None)

    def bwd(stats=P, logp=P, ent=P, g2=P, T=1.0, N=64, nbytes=1 << 40):
        o = lce.make_opts()
        return lib.lce_logprobs_keep_backward(P, P, P, N, 64, 1000, T, logp, stats, ent, P, g2, None, 0, P, P,
                                              ctypes.byref(o), P, nbytes, None)

    for rc in (fwd(stats=None), fwd(lse=None), bwd(stats=None), bwd(logp=None), bwd(ent=None), bwd(T=9e-7)):
        assert rc == E.LCE_ERR_INVALID_ARG
    for rc in (fwd(stats=P + 4), fwd(kept=P + 4), bwd(stats=P + 4), bwd(g2=P + 1)):
        assert rc == E.LCE_ERR_ALIGNMENT
    assert fwd(nbytes=lce.lce_logprobs_workspace_size(64, 64, 1000, 0) - 1) == E.LCE_ERR_WORKSPACE
    assert bwd(nbytes=lce.lce_logprobs_backward_workspace_size(64, 64, 1000) - 1) == E.LCE_ERR_WORKSPACE
    torch = pytest.importorskip("torch")
    f = torch.zeros(4)
    H, W, y = torch.zeros(4, 8).bfloat16(), torch.zeros(3, 8).bfloat16(), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: lce.lce_logprobs_keep(H, W, y), lambda: lce.lce_logprobs_keep_backward(H, W, y, f, f, f, f)):
        with pytest.raises(ValueError, match="CUDA tensors"):
            call()
    if not torch.cuda.is_available():   # these get as far as the device check
        for rc in (fwd(), bwd(), bwd(T=1e-6), fwd(N=0, stats=None), bwd(N=0, stats=None)):
            assert rc in (E.LCE_ERR_CUDA, E.LCE_ERR_UNSUPPORTED_DEVICE)


def test_a_frozen_head_needs_no_room_for_its_gradient(lib, monkeypatch):
    """Without dW neither the C calls nor the binding want the fp32 sum of a bf16 dW over the chunks."""
    E, P, o = lce, FAKE, lce.make_opts(chunk_tokens=32)
    small, large = [lce.lce_logprobs_backward_workspace_size(64, 64, 1000, g, o) for g in (0, E.LCE_DW_BF16)]
    kd_small, kd_large = [lce.lce_distill_workspace_size(64, 64, 1000, 5, True, g, o) for g in (0, E.LCE_DW_BF16)]
    assert large - small >= 4 * 1000 * 64 and kd_large - kd_small >= 4 * 1000 * 64

    def bwd(dW, nbytes):
        return lib.lce_logprobs_backward(P, P, P, 64, 64, 1000, 1.0, P, P, P, P, P, None, E.LCE_DW_BF16, P, dW,
                                         ctypes.byref(o), P, nbytes, None)

    def kd(dW, nbytes):
        return lib.lce_distill_fwd_bwd(P, P, P, P, 64, 64, 1000, 5, 0, 1.0, None, E.LCE_DW_BF16, P, P, P, dW,
                                       ctypes.byref(o), P, nbytes, None)

    assert bwd(P, small) == kd(P, kd_small) == E.LCE_ERR_WORKSPACE
    assert bwd(None, small - 1) == kd(None, kd_small - 1) == E.LCE_ERR_WORKSPACE
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():   # these get as far as the device check
        for rc in (bwd(P, large), kd(P, kd_large), bwd(None, small), kd(None, kd_small)):
            assert rc in (E.LCE_ERR_CUDA, E.LCE_ERR_UNSUPPORTED_DEVICE)
    asked = []
    monkeypatch.setattr(lce, "lce_logprobs_backward_workspace_size", lambda N, d, V, grads, o: asked.append(grads) or 0)
    H, W, f = torch.zeros(4, 8).bfloat16(), torch.zeros(3, 8).bfloat16(), torch.zeros(4)
    for need_dW in (True, False):
        with pytest.raises(lce.LCEError):   # a size of 0 ends the call
            lce._logprobs_backward(H, W, None, f, f, None, f, f, None, None, 1.0, E.LCE_DW_BF16, None, True, need_dW,
                                   None, None, {})
    assert asked == [E.LCE_DW_BF16, 0]


# --------------------------------------------------------------------------- the autograd modules, on fakes of the calls
@pytest.fixture
def fakes(monkeypatch):
    """The binding's calls replaced by ones that record themselves and return tensors of the right shapes."""
    torch = pytest.importorskip("torch")
    seen = []

    def logprobs(H, W, y, *, temperature=1.0, logits=None, **kw):
        seen.append(("logprobs", logits is not None))
        return tuple(torch.zeros(len(H)) for _ in range(3)) + (None, None)

    def logprobs_keep(H, W, y, **kw):
        return logprobs(H, W, y, **kw) + (torch.zeros(len(H), 2),)

    def logprobs_backward(H, W, *args):
        seen.append(("logprobs_backward",))
        return torch.zeros_like(H), torch.zeros_like(W)

    def distill_forward(H, W, idx, t, **kw):
        seen.append(("distill_forward",))
        return torch.zeros(1), torch.zeros(len(H))

    def distill_fwd_bwd(H, W, idx, t, *, need_dH=True, need_dW=True, **kw):
        seen.append(("distill_fwd_bwd", need_dH, need_dW))
        return (torch.zeros(1), torch.zeros(len(H)), torch.zeros_like(H) if need_dH else None,
                torch.zeros_like(W) if need_dW else None)

    monkeypatch.setattr(lce, "lce_logprobs", logprobs)
    monkeypatch.setattr(lce, "lce_logprobs_keep", logprobs_keep)
    monkeypatch.setattr(lce, "_logprobs_backward", logprobs_backward)
    monkeypatch.setattr(lce, "lce_distill_forward", distill_forward)
    monkeypatch.setattr(lce, "lce_distill_fwd_bwd", distill_fwd_bwd)
    monkeypatch.setattr(lce, "lce_scale_grads_bfloat", lambda dH, dW, g: None)
    H = torch.zeros(4, 8, dtype=torch.bfloat16, requires_grad=True)
    W = torch.zeros(30, 8, dtype=torch.bfloat16, requires_grad=True)
    return seen, H, W, torch.zeros(4, dtype=torch.int64), torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2)


@pytest.mark.parametrize("mode", ["no_grad", "inference_mode"])
def test_modules_without_grad_mode_run_the_forward_alone(fakes, mode):
    """Trainable tensors, but no graph: nothing is kept for a backward and no gradient computed."""
    import torch

    from chunked_lm_head_linear_gb300.autograd import FusedLinearDistillation, FusedLinearLogProbs
    seen, H, W, y, idx, t = fakes
    with getattr(torch, mode)():
        logp, ent = FusedLinearLogProbs(recompute=False)(H, W, y)
        loss = FusedLinearDistillation()(H, W, idx, t)
    assert not (logp.requires_grad or ent.requires_grad or loss.requires_grad)
    assert seen == [("logprobs", False), ("distill_forward",)]
    del seen[:]
    FusedLinearLogProbs(recompute=False)(H, W, y)
    FusedLinearDistillation()(H, W.detach(), idx, t)
    assert seen == [("logprobs", True), ("distill_fwd_bwd", True, False)]


def test_what_the_forward_keeps_is_freed_by_the_backward(fakes):
    """The kept logits are saved tensors: freed with the graph's other ones, though an output lives on."""
    import weakref

    import torch

    from chunked_lm_head_linear_gb300.autograd import FusedLinearLogProbs
    _, H, W, y, _, _ = fakes
    kept = []
    keep = lce.lce_logprobs_keep
    lce.lce_logprobs_keep = lambda *a, **kw: (kept.append(weakref.ref(kw["logits"])), keep(*a, **kw))[1]   # fakes undoes it
    logp, _ = FusedLinearLogProbs(recompute=False)(H, W, y)
    torch.autograd.grad(logp.sum(), [H, W], retain_graph=True)
    assert kept[0]() is not None
    torch.autograd.grad(logp.sum(), [H, W])
    assert kept[0]() is None


@pytest.mark.parametrize("N,d,chunk,kept", [(64, 1024, 0, False), (64, 1536, 0, True), (6143, 1536, 0, True),
                                            (6144, 1536, 0, False), (65, 2048, 64, False), (64, 2048, 64, True),
                                            (64, 2048, "auto", False)])
def test_which_logits_are_kept(fakes, N, d, chunk, kept):
    """recompute=None: those of a batch of one chunk, from d = 1536 on."""
    import torch

    from chunked_lm_head_linear_gb300.autograd import FusedLinearLogProbs
    seen, _, _, _, _, _ = fakes
    H, W = torch.zeros(N, d, dtype=torch.bfloat16, requires_grad=True), torch.zeros(9, d, dtype=torch.bfloat16)
    FusedLinearLogProbs(chunk_tokens=chunk)(H, W, torch.zeros(N, dtype=torch.int64))
    assert seen == [("logprobs", kept)]
