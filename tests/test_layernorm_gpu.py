"""Layer norm where its persistent blocks take many turns of their ring, for every class of row length, and where no cluster
is used, whole outputs against fp64 on the device. Tolerances: those of test_losses_gpu.py (g = (d / 32 + 16) eps and so on)."""
import ctypes

import pytest

from test_tokens_gpu import U

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


def _torch():
    import torch
    return torch


def inputs(N, d, f32_x, seed=0):
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = rand(N, d) * (0.5 + 4.0 * torch.rand(N, 1, generator=g, device="cuda")) + 0.5
    return x if f32_x else x.bfloat16(), 1 + 0.3 * rand(d), rand(d), rand(N, d).bfloat16()


def within(got, ref, tol, what):
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), f"{what}: off by {err.max().item():.3e}, {(err / tol).max().item():.2f} of the bound"


def check(x, w, b, dH, eps, H=None, mean=None, rstd=None, dx=None, dw=None, db=None):
    """What is given, against the definition in fp64."""
    N, d = x.shape
    X, G, w64, b64 = x.double(), dH.double(), w.double(), b.double()
    mu = X.mean(1, keepdim=True)
    r = 1 / ((X - mu).square().mean(1, keepdim=True) + float(eps)).sqrt()
    xh = (X - mu) * r
    g = (d / 32 + 16) * EPS
    em = g * X.abs().mean(1, keepdim=True) + 2.0 ** -149
    rel = 2 * g + (em * r).square() + 2.0 ** -21
    ex = r * em + xh.abs() * rel
    if H is not None:
        want = xh * w64 + b64
        within(mean, mu[:, 0], (em + EPS * mu.abs())[:, 0], "mean")
        within(rstd, r[:, 0], (r * rel)[:, 0], "rstd")
        within(H, want, (w64.abs() * ex + 2.0 ** -21 * (xh * w64).abs() + 2.0 ** -21 * b64.abs()) * (1 + U) + U * want.abs(), "H")
    if dx is not None:
        gw = G * w64
        c = (gw * xh).mean(1, keepdim=True)
        want = r * (gw - gw.mean(1, keepdim=True) - xh * c)
        bulk = r * (gw.abs() + gw.abs().mean(1, keepdim=True) + xh.abs() * (gw * xh).abs().mean(1, keepdim=True))
        tol = (3 * g + 2.0 ** -20 + rel) * bulk + r * (ex * c.abs() + xh.abs() * (gw.abs() * ex).mean(1, keepdim=True))
        within(dx, want, tol * (1 + U) + (U * want.abs() if dx.dtype == _torch().bfloat16 else 0) + 1e-38, "dx")
    if dw is not None:
        within(dw, (G * xh).sum(0), (G.abs() * ex).sum(0) + (N * EPS + 2.0 ** -21) * (G * xh).abs().sum(0) + 1e-38, "dw")
    if db is not None:
        within(db, G.sum(0), (N * EPS + 2.0 ** -21) * G.abs().sum(0) + 1e-38, "db")


# More rows than all blocks hold in all turns of their rings, and a last turn that is not full
@pytest.mark.parametrize("N,d", [(60013, 8), (40001, 200), (31999, 256), (12001, 264), (11003, 512), (7001, 520), (6501, 1024),
                                 (5003, 1032), (3001, 2048), (2707, 2056), (2501, 4096), (1603, 4104), (1201, 8192), (801, 8200),
                                 (653, 16384), (455, 32768)])
@pytest.mark.parametrize("f32_x", [False, True])
def test_many_turns(cuda_lib, N, d, f32_x):
    torch = _torch()
    x, w, b, dH = inputs(N, d, f32_x, seed=d)
    H, mean, rstd = cuda_lib.lce_layernorm_forward(x, w, b, 1e-5)
    eps = torch.tensor(1e-5).item()
    check(x, w, b, dH, eps, H, mean, rstd)
    dx, dw, db = cuda_lib.lce_layernorm_backward(x, w, mean, rstd, dH)
    check(x, w, b, dH, eps, dx=dx, dw=dw, db=db)
    # dx alone (no sums), dw and db alone (no exchange in a row), db alone
    assert torch.equal(cuda_lib.lce_layernorm_backward(x, w, mean, rstd, dH, need_dw=False, bias=False)[0], dx)
    _, dw2, db2 = cuda_lib.lce_layernorm_backward(x, w, mean, rstd, dH, need_dx=False)
    assert torch.equal(dw2, dw) and torch.equal(db2, db)
    assert torch.equal(cuda_lib.lce_layernorm_backward(x, w, mean, rstd, dH, need_dx=False, need_dw=False)[2], db)


@pytest.mark.parametrize("N,d", [(0, 64), (1, 8), (1, 8192), (3, 24), (65, 256), (300, 264), (1531, 264), (33, 520), (500, 1000),
                                 (200, 2048), (17, 2056), (128, 4096), (9, 4104), (64, 8192)])
@pytest.mark.parametrize("f32_x", [False, True])
def test_backward_where_no_cluster_fits(cuda_lib, N, d, f32_x):
    """Small backward calls are one cluster of sixteen blocks; where the device has no room for one they take the launches of
    large calls, in the same workspace, and leave what lies behind it alone."""
    torch = _torch()
    x, w, b, dH = inputs(N, d, f32_x, seed=N + d)
    _, mean, rstd = cuda_lib.lce_layernorm_forward(x, w, b)
    need = cuda_lib.lce_layernorm_workspace_size(N, d)
    p = lambda t: ctypes.c_void_p(0 if t is None else t.data_ptr())  # noqa: E731
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    kind = cuda_lib.LCE_NORM_X_F32 if f32_x else 0
    got = []
    for types in (kind, kind | cuda_lib.LCE_TEST_NO_CLUSTER):
        ws = torch.full((need + 256,), 7, dtype=torch.uint8, device="cuda")
        dx, dw, db = torch.full_like(x, 3.0), torch.full_like(w, 3.0), torch.full_like(w, 3.0)
        rc = cuda_lib.load().lce_layernorm_backward(p(x), p(w), p(mean), p(rstd), p(dH), N, d, types, p(dx), p(dw), p(db),
                                                    p(ws), need, stream)
        assert rc == 0 and bool((ws[need:] == 7).all())
        check(x, w, b, dH, torch.tensor(1e-5).item(), dx=dx, dw=dw, db=db)
        got.append(dx)
    assert torch.equal(*got)


def test_the_test_value_is_refused_elsewhere(cuda_lib):
    x = _torch().zeros(4, 64, device="cuda")
    p = ctypes.c_void_p(x.data_ptr())
    rc = cuda_lib.load().lce_layernorm_forward(p, None, None, 2, 64, 1e-5, cuda_lib.LCE_NORM_X_F32 | cuda_lib.LCE_TEST_NO_CLUSTER,
                                               p, None, None, None)
    assert rc == cuda_lib.LCE_ERR_INVALID_ARG
