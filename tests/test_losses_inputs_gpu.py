"""The policy and preference losses on hidden states and weights as a model gives them (normally distributed bf16), whose
logits no fp32 sum has exactly; against the other operators of the head, and against fp64 on the device.

Tolerances, eps = 2^-24, u = 2^-8, x the largest |z_v - m| of the row over T:
  between operators  both take the logits from the same GEMM. On either side a term exp(x) errs by the roundings of its
                     argument, 3 eps x, and 2^-22 (ex2.approx); its sum runs through 32 terms, 4 groups and 40 merges of
                     half tiles, and logp's own operations add 8 eps (|logp| + 2): (3 x + 4 + 76 + 8 (|logp| + 2)) eps a side
  against fp64       the GEMM adds d / 16 partial products into an fp32 that may be cut instead of rounded: each step
                     2^-23 of the sum so far, which is at most the row's sum of |h w| =: s; so a logit errs by
                     tz = (d / 16) 2^-23 s at most, logp by 2 tz / T and the above
  gradients          p errs by 2 tz relative; entries and scales as in test_losses_gpu.py (exp tiles)
"""
import numpy as np
import pytest

from test_losses_gpu import uses_exp_tiles
from test_tokens_gpu import U

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


def _torch():
    import torch
    return torch


def model_inputs(N, d, V, peak=14.0, seed=0):
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = (torch.randn(V, d, generator=g, device="cuda") * 0.02).bfloat16()
    y = torch.randint(0, V, (N,), generator=g, device="cuda")
    lean = peak * torch.rand(N, 1, generator=g, device="cuda") / (0.0004 * d)
    H = (torch.randn(N, d, generator=g, device="cuda") + W[y].float() * lean).bfloat16()
    y[::9] = -100
    return g, H, W, y


@pytest.mark.parametrize("N,d,V,T", [(300, 2048, 40001, 1.0), (300, 7168, 40001, 1.0), (300, 7168, 40001, 0.5),
                                     (100, 4096, 100003, 1.0), (200, 7168, 4099, 1.0)])
def test_losses_of_a_models_hidden_states(cuda_lib, N, d, V, T):
    torch = _torch()
    g, H, W, y = model_inputs(N, d, V, seed=d)
    told = y >= 0
    at = torch.where(told, y, 0)[:, None]
    A = torch.randn(N, generator=g, device="cuda")
    cu = torch.tensor([0, N // 3, N // 2, N - 20, N - 1], device="cuda")
    kw = dict(temperature=T, sync_check=True)
    loss, logp, row, dH, dW = cuda_lib.lce_policy_fwd_bwd(H, W, y, A, dW_dtype=torch.bfloat16, **kw)
    other = cuda_lib.lce_logprobs(H, W, y, temperature=T)[0]
    forward = cuda_lib.lce_policy_forward(H, W, y, A, temperature=T)[1]
    seq = cuda_lib.lce_preference_fwd_bwd(H, W, y, cu, **kw)[2]
    z = H.double() @ W.double().t() / T
    far = (z.amax(1) - z.amin(1)).clamp_min(1.0)
    e = torch.exp(z - z.gather(1, at)).scatter_(1, at, 0.0)
    rest = e.sum(1)
    want = torch.where(told, -torch.log1p(rest), 0.0)
    side = (3 * far + 80 + 8 * (want.abs() + 2)) * EPS
    for got, name in ((logp, "policy step"), (forward, "policy loss")):
        assert ((got - other).abs() <= 2 * side).all(), (name, ((got - other).abs() / side).max().item())
    for s in range(4):
        rows = slice(int(cu[s]), int(cu[s + 1]))
        assert (seq[s].double() - other[rows].double().sum()).abs() <= 2 * side[rows].sum() + 2 * EPS * want[rows].abs().sum()
    # a ratio to the same model's log-probabilities is 1
    ratio = cuda_lib.lce_policy_fwd_bwd(H, W, y, torch.ones_like(A), other, clip_low=0.0, clip_high=0.0, **kw)[2]
    assert ((ratio + told.float()).abs() <= 2 * side + 2 * EPS).all()
    s = (H.double().abs() @ W.double().abs().t()).amax(1)
    tz = (d / 16) * 2.0 ** -23 * s / T
    assert ((logp - want).abs() <= 2 * tz + side).all(), ((logp - want).abs() / (2 * tz + side)).max().item()
    # gradients, at columns of both ends
    a = torch.where(told, -A.double(), 0.0)[:, None] / int(told.sum()) / T
    p = e / (1 + rest)[:, None]
    G = (-p).scatter_(1, at, (rest / (1 + rest))[:, None]) * a
    size = G.abs()
    exp = 1 if uses_exp_tiles(N, V, 0) else 0
    slack = (2 * tz + 2.0 ** -10)[:, None]
    want_dH, bulk = G @ W.double(), size @ W.double().abs()
    assert ((dH - want_dH).abs() <= ((1 + U) ** (1 + exp) - 1 + slack) * bulk + U * want_dH.abs() + 1e-30).all()
    cols = torch.tensor([0, 127, 128, 255, 256, V // 2, V - 130, V - 2, V - 1, *np.unique(y[told][:5].cpu())], device="cuda")
    want_dW = G[:, cols].t() @ H.double()
    bulk = ((1 + U) ** (2 + exp) - 1 + slack) * size[:, cols]
    assert ((dW[cols] - want_dW).abs() <= bulk.t() @ H.double().abs() + U * want_dW.abs() + 1e-30).all()
    for got, ref in ((dH, want_dH), (dW[cols], want_dW)):
        assert (got - ref).norm() <= 5e-3 * ref.norm()


@pytest.mark.parametrize("N,d,V,chunk", [(40, 256, 151936, 0), (300, 2048, 100003, 0), (600, 1032, 100003, 256), (200, 264, 4099, 0)])
def test_a_frozen_head(cuda_lib, N, d, V, chunk):
    """dH alone, whose launch cuts the vocabulary otherwise than one with dW does: against fp64, in a workspace of the size
    asked for, and nothing behind it touched. The bound on dH as above; sums of up to 32 parts add 32 eps of the terms."""
    torch = _torch()
    g, H, W, y = model_inputs(N, d, V, seed=d)
    told = y >= 0
    at = torch.where(told, y, 0)[:, None]
    A = torch.randn(N, generator=g, device="cuda")
    cu = torch.tensor([0, N // 3, N - 1], device="cuda")
    opts = cuda_lib.make_opts(chunk_tokens=chunk)
    z = H.double() @ W.double().t()
    e = torch.exp(z - z.gather(1, at)).scatter_(1, at, 0.0)
    rest = e.sum(1)
    unit = (-e / (1 + rest)[:, None]).scatter_(1, at, (rest / (1 + rest))[:, None])
    tz = (d / 16) * 2.0 ** -23 * (H.double().abs() @ W.double().abs().t()).amax(1)
    exp = 1 if uses_exp_tiles(N, V, chunk) else 0
    for name, size, args in (("policy", cuda_lib.lce_policy_workspace_size(N, d, V, True, 0, opts), (A,)),
                             ("preference", cuda_lib.lce_preference_workspace_size(N, d, V, 1, True, 0, opts), (cu,))):
        ws = torch.full((size + 4096,), 9, dtype=torch.uint8, device="cuda")
        call = getattr(cuda_lib, f"lce_{name}_fwd_bwd")
        out = call(H, W, y, *args, need_dW=False, workspace=ws[:size], chunk_tokens=chunk, sync_check=True)
        assert out[4] is None and bool((ws[size:] == 9).all())
        again = call(H, W, y, *args, need_dW=False, chunk_tokens=chunk)
        assert torch.equal(out[3], again[3])
        if name == "policy":
            a = torch.where(told, -A.double() / int(told.sum()), 0.0)
        else:   # sigmoid, beta = 0.1, one pair: the slope from the sums that came out
            slope = -0.1 * torch.sigmoid(-0.1 * (out[2][0] - out[2][1]).double())
            a = torch.zeros(N, dtype=torch.float64, device="cuda")
            a[:N // 3], a[N // 3:N - 1] = slope, -slope
            a = torch.where(told, a, 0.0)
        G = unit * a[:, None]
        want, bulk = G @ W.double(), G.abs() @ W.double().abs()
        slack = (2 * tz + 2.0 ** -10 + 32 * EPS)[:, None]
        assert ((out[3] - want).abs() <= ((1 + U) ** (1 + exp) - 1 + slack) * bulk + U * want.abs() + 1e-30).all()
        # a pair hundreds of nats apart has a slope below the least normal number of fp32 and bf16, 2^-126: such elements may be 0
        assert (out[3] - want).norm() <= 5e-3 * want.norm() + 2.0 ** -126 * want.numel() ** 0.5


def test_coldest_temperature_with_two_sums_of_a_logit(cuda_lib):
    """Logits of thousands at T = 1e-6: the label's two sums lie hundreds of nats apart, and the exact tiles take over. With the
    label the row's largest logit it has all of the probability (log 1 = 0, no gradient), else it has none of it."""
    torch = _torch()
    N, d, V, T = 300, 2048, 40001, 1.0e-6
    g, H, W, y = model_inputs(N, d, V, seed=3)
    H = (H.float() * 60).bfloat16()
    other = cuda_lib.lce_logprobs(H, W, torch.zeros_like(y), temperature=T, top_k=2)
    gap = (other[3][:, 0] - other[3][:, 1])
    y = torch.where(gap > 1.0e3, other[4][:, 0], -100)
    assert int((y >= 0).sum()) > N // 2
    y[0] = other[4][0, 1]
    A = torch.randn(N, generator=g, device="cuda")
    loss, logp, row, dH, dW = cuda_lib.lce_policy_fwd_bwd(H, W, y, A, temperature=T, dW_dtype=torch.bfloat16, sync_check=True)
    want = cuda_lib.lce_logprobs(H, W, y, temperature=T)[0]
    assert torch.equal(logp[1:], torch.zeros_like(logp[1:])) and not dH[1:].any()
    assert logp[0] == want[0] < -1.0e3 and torch.isfinite(dH).all() and torch.isfinite(dW.float()).all()
    told = y >= 0
    assert ((row + torch.where(told, A, 0.0)).abs() <= 2 * EPS * A.abs()).all() and torch.isfinite(loss).all()
