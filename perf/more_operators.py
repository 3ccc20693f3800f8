"""Losses of policy and preference training on the LM head, and the layer norm
in front of it, as a user's program calls them, with their plain forms.

norm        layer norm of the last hidden states, alone or with its gradients
policy      clipped policy loss with a KL term, loss alone or with gradients
preference  loss of paired sequences' log ratios, with gradients

The head takes hidden states H [N, d] and W [V, d] in bf16. As in operators.py
their values lie on a coarse grid, so that logits are exact in fp32 whatever the
order of their sum. What the losses compare with a border (a ratio with the
clipping range, a margin with the hinge) keeps a distance to it, as the gradient
jumps there.
"""
import math

import torch

own = False

IGNORE = -100


def listed():
    return [
        # the last norm of one decoded token
        dict(name="norm_decode_1", op="norm", N=1, d=2048, x="bf16", bias=True, grad=False),
        # a prompt's hidden states held in fp32, no bias
        dict(name="norm_prompt_8192", op="norm", N=8192, d=2048, x="fp32", bias=False, grad=False),
        # a training step, small odd sizes
        dict(name="norm_train_odd_1531", op="norm", N=1531, d=264, x="bf16", bias=False, grad=True),
        # a training step over a long packed batch
        dict(name="norm_train_65536", op="norm", N=65536, d=4096, x="bf16", bias=True, grad=True),
        # a small policy, latency-bound
        dict(name="policy_odd_250", op="policy", N=250, d=264, V=4099, T=0.9, kl="k3", old=True, dual=0.0,
             weights=False, grad=True),
        # one micro-batch, sampled by the model as it is
        dict(name="policy_1024", op="policy", N=1024, d=2048, V=151936, T=1.0, kl="none", old=False, dual=0.0,
             weights=True, grad=True),
        # a wider head over a longer batch, every term
        dict(name="policy_4096", op="policy", N=4096, d=4096, V=151936, T=1.0, kl="k3", old=True, dual=3.0,
             weights=True, grad=True),
        # the loss on held-out samples
        dict(name="policy_eval_1531", op="policy", N=1531, d=2048, V=151655, T=0.7, kl="k2", old=True, dual=0.0,
             weights=False, grad=False),
        # two short pairs of a small model
        dict(name="preference_tiny_300", op="preference", N=300, d=256, V=4096, pairs=2, kind="hinge", mean=False,
             ref=True),
        # one micro-batch of pairs
        dict(name="preference_2048", op="preference", N=2048, d=2048, V=151936, pairs=4, kind="sigmoid", mean=False,
             ref=True),
        # a packed batch longer than a chunk, no reference model, lengths averaged
        dict(name="preference_9000", op="preference", N=9000, d=2048, V=151936, pairs=9, kind="sigmoid", mean=True,
             ref=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "policy", "policy", "preference"])
    if op == "norm":
        while True:
            N, d = _log(rng, 1, 65536), 8 * _log(rng, 8, 1024)
            if N * d <= 65536 * 4096:
                break
        return dict(op=op, N=N, d=d, x=rng.choice(["bf16", "fp32"]), bias=rng.random() < 0.5, grad=rng.random() < 0.6)
    while True:
        N, d, V = _log(rng, 64, 9000), 8 * _log(rng, 256 // 8, 4096 // 8), _log(rng, 1000, 151936)
        if N * d * V <= 9000 * 2048 * 151936:
            break
    if op == "policy":
        return dict(op=op, N=N, d=d, V=V, T=rng.choice([1.0, 1.0, 0.7, 1.2]), kl=rng.choice(["none", "k1", "k2", "k3"]),
                    old=rng.random() < 0.7, dual=rng.choice([0.0, 3.0]), weights=rng.random() < 0.5,
                    grad=rng.random() < 0.8)
    return dict(op=op, N=N, d=d, V=V, pairs=rng.randint(1, max(1, N // 64)), kind=rng.choice(["sigmoid", "hinge", "ipo"]),
                mean=rng.random() < 0.4, ref=rng.random() < 0.7)


EPS = 1e-5
CLIP = (0.2, 0.28)       # how far a ratio may fall and rise
KL_COEF = 0.04
MARGIN = 0.5             # sigmoid and hinge without a reference


def _beta(case):
    """Averaged log ratios are small, so their factor is large."""
    return 2.0 if case["mean"] else 0.1


def _grid(x, steps):
    return (x * steps).round_().clamp_(-127, 127).div_(steps).to(torch.bfloat16)


def _away(x, border, gap):
    """x, at least gap from border."""
    return torch.where((x - border).abs() < gap, border + torch.where(x < border, -gap, gap), x)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    N, d = case["N"], case["d"]
    s = dict(case=dict(case))
    if case["op"] == "norm":
        dtype = torch.bfloat16 if case["x"] == "bf16" else torch.float32
        s["x"] = randn(N, d).mul_(4.0 * rand(N, 1) + 0.5).add_(0.3 * randn(d)).to(dtype)   # rows of other sizes
        s["w"] = 1.0 + 0.2 * randn(d)
        s["b"] = 0.1 * randn(d) if case["bias"] else None
        if case["grad"]:
            s["dH"] = (randn(N, d) * rand(N, 1)).to(torch.bfloat16)
        return s
    V = case["V"]
    sigma = 0.02 if d <= 2048 else 0.015
    W = _grid(randn(V, d).mul_(sigma), 1024.0)
    y = (rand(N).pow(2) * V).long().clamp_(max=V - 1)   # low ids are the frequent ones
    H = _grid(randn(N, d).add_(W[y].float() * (16.0 * rand(N, 1) / (sigma * sigma * d))), 16.0)
    s.update(H=H, W=W)
    T = case.get("T", 1.0)
    logp = torch.empty(N, device="cuda")                # what the model gives the tokens
    for r in range(0, N, 2048):
        z = H[r:r + 2048].float() @ W.float().t() / T
        logp[r:r + 2048] = z.gather(1, y[r:r + 2048, None])[:, 0] - torch.logsumexp(z, 1)
    if case["op"] == "policy":
        given = rand(N) >= 0.1                          # the others are prompts and padding
        sequence = torch.cumsum((rand(N) < 1 / 256).long(), 0)
        s["advantages"] = randn(N)[sequence].contiguous()   # one of each sampled answer
        step = 0.25 * randn(N)                          # log ratio to the policy that sampled
        for border in (1 - CLIP[0], 1 + CLIP[1], 3.0):
            step = _away(step, math.log(border), 1e-3)
        s["old"] = torch.where(given, logp - step, 0.0) if case["old"] else None
        s["ref"] = torch.where(given, logp - 0.5 * randn(N), 0.0) if case["kl"] != "none" else None
        s["weights"] = None
        if case["weights"]:                             # every answer counts the same
            length = torch.bincount(sequence, weights=given.float()).clamp(min=1.0)
            s["weights"] = (N / length[sequence] / (sequence[-1] + 1)).float().contiguous()
        s["y"] = torch.where(given, y, IGNORE)
        return s
    S = 2 * case["pairs"]
    used = N - int(0.05 * N)                            # rows behind the last sequence are padding
    length = torch.cumsum(0.2 + rand(S), 0)
    cu = torch.cat([torch.zeros(1, device="cuda"), length / length[-1] * used]).round().long()
    cu[-1] = used
    i = torch.arange(N, device="cuda")
    seq = torch.searchsorted(cu, i, right=True) - 1     # S and beyond: padding
    prompt = (i - cu[seq.clamp(max=S)]) < 0.25 * (cu[(seq + 1).clamp(max=S)] - cu[seq.clamp(max=S)])
    s["y"] = torch.where(prompt | (i >= used), IGNORE, y)
    s["cu"] = cu
    s["ref"] = None
    total, _ = _sums(s, logp.double())
    beta = _beta(case)
    if case["ref"]:
        x = _away(0.5 + 1.5 * randn(case["pairs"]), 1.0, 0.02).double()
        ref = total + randn(S) / beta
        ref[0::2] += (total[0::2] - ref[0::2]) - (total[1::2] - ref[1::2]) - x / beta
        s["ref"] = ref.float()
    return s


def _sums(s, logp):
    """Log-probability of each sequence: the sum over its given tokens, or their mean; and the factor of a token in it."""
    cu, told = s["cu"], s["y"] != IGNORE
    S = cu.numel() - 1
    i = torch.arange(logp.numel(), device=cu.device)
    seq = (torch.searchsorted(cu, i, right=True) - 1).clamp(max=S - 1)
    told = told & (i >= cu[0]) & (i < cu[-1])
    total = torch.zeros(S, dtype=logp.dtype, device=cu.device).index_add_(0, seq, torch.where(told, logp, 0.0))
    count = torch.zeros(S, dtype=logp.dtype, device=cu.device).index_add_(0, seq, told.to(logp.dtype)).clamp(min=1)
    if s["case"]["mean"]:
        return total / count, told / count[seq]
    return total, told.to(logp.dtype)


def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own_norm(s):
    from chunked_lm_head_linear_gb300 import lce
    H, mean, rstd = lce.lce_layernorm_forward(s["x"], s["w"], s["b"], eps=EPS)
    if not s["case"]["grad"]:
        return dict(H=H)
    dx, dw, db = lce.lce_layernorm_backward(s["x"], s["w"], mean, rstd, s["dH"], bias=s["b"] is not None)
    return dict(H=H, dx=dx, dw=dw, db=db)


def _own_policy(s):
    from chunked_lm_head_linear_gb300 import lce
    c = s["case"]
    kw = dict(weights=s["weights"], temperature=c["T"], clip_low=CLIP[0], clip_high=CLIP[1], dual_clip=c["dual"])
    if c["kl"] != "none":
        kw.update(kl=c["kl"], kl_coef=KL_COEF)
    args = s["H"], s["W"], s["y"], s["advantages"], s["old"], s["ref"]
    if not c["grad"]:
        loss, logp, row_loss = lce.lce_policy_forward(*args, **kw)
        return dict(loss=loss, logp=logp, row_loss=row_loss)
    loss, logp, row_loss, dH, dW = lce.lce_policy_fwd_bwd(*args, dW_dtype=torch.bfloat16, **kw)
    return dict(loss=loss, logp=logp, row_loss=row_loss, dH=dH, dW=dW)


def _own_preference(s):
    from chunked_lm_head_linear_gb300 import lce
    c = s["case"]
    loss, pair_loss, seq_logp, dH, dW = lce.lce_preference_fwd_bwd(
        s["H"], s["W"], s["y"], s["cu"], s["ref"], kind=c["kind"], beta=_beta(c), margin=_margin(c), average=c["mean"],
        dW_dtype=torch.bfloat16)
    return dict(loss=loss, pair_loss=pair_loss, seq_logp=seq_logp, dH=dH, dW=dW)


def _margin(c):
    return 0.0 if c["ref"] or c["kind"] == "ipo" else MARGIN


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + EPS)
    xh = (x - mean) * rstd
    H = xh * s["w"]
    if s["b"] is not None:
        H = H + s["b"]
    H = H.bfloat16()
    if not s["case"]["grad"]:
        return dict(H=H)
    dH = s["dH"].float()
    g = dH * s["w"]
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dict(H=H, dx=dx.to(s["x"].dtype), dw=(dH * xh).sum(0), db=dH.sum(0) if s["b"] is not None else None)


def _head(s, T):
    """H and W in fp32, softmax and log-probabilities of the given tokens."""
    H, W = s["H"].float(), s["W"].float()
    z = (H @ W.t()).div_(T)
    z -= z.amax(1, keepdim=True)
    p = torch.exp(z)
    total = p.sum(1, keepdim=True)
    at = s["y"].clamp(min=0)[:, None]
    logp = (z.gather(1, at) - torch.log(total))[:, 0]
    return H, W, p.div_(total), at, logp


def _gradients(H, W, p, at, a):
    """dH and dW for a = dloss / dlogp over T."""
    G = p.mul_(-a[:, None])
    G.scatter_add_(1, at, a[:, None])
    return dict(dH=(G @ W).bfloat16(), dW=(G.t() @ H).bfloat16())


def _plain_policy(s):
    c, given = s["case"], s["y"] != IGNORE
    H, W, p, at, logp = _head(s, c["T"])
    l, A = logp.double(), s["advantages"].double()           # ratios next to a border
    r = torch.exp(l - s["old"].double()) if s["old"] is not None else torch.ones_like(l)
    free, bound = r * A, torch.clamp(r, 1 - CLIP[0], 1 + CLIP[1]) * A
    gain, slope = torch.where(free <= bound, free, bound), torch.where(free <= bound, free, 0.0)
    if c["dual"] > 0:
        far = (A < 0) & (gain < c["dual"] * A)
        gain, slope = torch.where(far, c["dual"] * A, gain), torch.where(far, 0.0, slope)
    row, a = -gain, -slope
    if c["kl"] != "none":
        u = l - s["ref"].double()
        kl, dkl = {"k1": (u, torch.ones_like(u)), "k2": (u * u / 2, u),
                   "k3": (torch.exp(-u) - 1 + u, 1 - torch.exp(-u))}[c["kl"]]
        row, a = row + KL_COEF * kl, a + KL_COEF * dkl
    if s["weights"] is not None:
        row, a = row * s["weights"].double(), a * s["weights"].double()
    row = torch.where(given, row, 0.0)
    n = given.sum().clamp(min=1)
    out = dict(loss=(row.sum() / n).float().reshape(1), logp=torch.where(given, logp, 0.0), row_loss=row.float())
    if not c["grad"]:
        return out
    a = torch.where(given, a, 0.0) / (n * c["T"])
    return dict(out, **_gradients(H, W, p, at, a.float()))


def _plain_preference(s):
    c, beta = s["case"], _beta(s["case"])
    H, W, p, at, logp = _head(s, 1.0)
    total, factor = _sums(s, logp.double())                  # long sums
    delta = total[0::2] - total[1::2]
    if s["ref"] is not None:
        delta = delta - (s["ref"][0::2].double() - s["ref"][1::2].double())
    x = beta * delta - _margin(c)
    if c["kind"] == "sigmoid":
        pair = torch.clamp(-x, min=0) + torch.log1p(torch.exp(-x.abs()))
        slope = -beta / (1 + torch.exp(x))
    elif c["kind"] == "hinge":
        pair, slope = torch.clamp(1 - x, min=0), torch.where(x < 1, -beta, 0.0).to(x)
    else:
        pair = (delta - 1 / (2 * beta)).square()
        slope = 2 * (delta - 1 / (2 * beta))
    P, S = c["pairs"], 2 * c["pairs"]
    i = torch.arange(c["N"], device=total.device)
    seq = (torch.searchsorted(s["cu"], i, right=True) - 1).clamp(max=S - 1)
    a = torch.stack([slope, -slope], 1).reshape(-1)[seq] * factor / P
    out = dict(loss=(pair.sum() / P).float().reshape(1), pair_loss=pair.float(), seq_logp=total.float())
    return dict(out, **_gradients(H, W, p, at, a.float()))


_own = dict(norm=_own_norm, policy=_own_policy, preference=_own_preference)
_plain = dict(norm=_plain_norm, policy=_plain_policy, preference=_plain_preference)


def work(case):
    N, d = case["N"], case["d"]
    if case["op"] == "norm":
        size, extra = (2 if case["x"] == "bf16" else 4), 4 * d * (2 if case["bias"] else 1)
        if not case["grad"]:
            return dict(bytes=N * d * (size + 2) + extra, flops=8 * N * d)
        return dict(bytes=N * d * (2 * size + 4) + 2 * extra, flops=24 * N * d)   # x and dH read, H and dx written
    V = case["V"]
    rows = 2 * N * d + 2 * V * d + 8 * N
    if case["op"] == "policy":     # advantages, what else is given, logp and the rows' losses
        rows += 4 * N * (3 + case["old"] + case["weights"] + (case["kl"] != "none"))
    if not case.get("grad", True):
        return dict(bytes=rows, flops=2 * N * V * d)
    return dict(bytes=rows + 2 * N * d + 2 * V * d, flops=6 * N * V * d)


def exact(case, seed):
    """The definitions in 64 bits, the losses differentiated by autograd; None where the products would take too long."""
    if case["op"] == "norm":
        if case["N"] * case["d"] > 3e8:
            return None
        s = prepare(case, seed)
        x = s["x"].double().requires_grad_(True)
        w = s["w"].double().requires_grad_(True)
        centred = x - x.sum(1, keepdim=True) / case["d"]
        H = centred * w / torch.sqrt((centred * centred).sum(1, keepdim=True) / case["d"] + EPS)
        if s["b"] is not None:
            H = H + s["b"].double()
        if not case["grad"]:
            return dict(H=H.detach())
        dx, dw = torch.autograd.grad(H, [x, w], s["dH"].double())
        return dict(H=H.detach(), dx=dx, dw=dw, db=s["dH"].double().sum(0) if s["b"] is not None else None)
    if work(case)["flops"] > 5e12:
        return None
    s = prepare(case, seed)
    H, W, T, y, N = s["H"].double(), s["W"].double(), case.get("T", 1.0), s["y"], case["N"]
    logp = torch.zeros(N, dtype=torch.float64, device=H.device)
    blocks = [slice(r, min(N, r + 512)) for r in range(0, N, 512)]
    for b in blocks:
        logq = torch.log_softmax(H[b] @ W.t() / T, 1)
        told = (y[b] >= 0).nonzero()[:, 0]
        logp[b.start + told] = logq[told, y[b][told]]
    logp.requires_grad_(True)
    loss, out = (_exact_policy if case["op"] == "policy" else _exact_preference)(s, logp)
    if not case.get("grad", True):
        return out
    a = torch.autograd.grad(loss, logp)[0] / T
    dH, dW = torch.zeros_like(H), torch.zeros_like(W)
    for b in blocks:
        G = torch.softmax(H[b] @ W.t() / T, 1).mul_(-a[b, None])
        told = (y[b] >= 0).nonzero()[:, 0]
        G[told, y[b][told]] += a[b][told]
        dH[b] = G @ W
        dW += G.t() @ H[b]
    return dict(out, dH=dH, dW=dW)


def _exact_policy(s, logp):
    c = s["case"]
    told = (s["y"] >= 0).nonzero()[:, 0]
    l, A = logp[told], s["advantages"].double()[told]
    ratio = (l - (l.detach() if s["old"] is None else s["old"].double()[told])).exp()
    gain = torch.minimum(ratio * A, ratio.clamp(1 - CLIP[0], 1 + CLIP[1]) * A)
    if s["old"] is None:
        gain = ratio * A
    if c["dual"] > 0:
        gain = torch.where(A < 0, torch.maximum(gain, c["dual"] * A), gain)
    row = -gain
    if c["kl"] != "none":
        u = l - s["ref"].double()[told]
        row = row + KL_COEF * (u if c["kl"] == "k1" else u.square() / 2 if c["kl"] == "k2" else torch.expm1(-u) + u)
    if s["weights"] is not None:
        row = row * s["weights"].double()[told]
    loss = row.sum() / max(len(told), 1)
    rows = torch.zeros_like(logp).index_put((told,), row).detach()
    return loss, dict(loss=loss.detach().reshape(1), logp=logp.detach(), row_loss=rows)


def _exact_preference(s, logp):
    c, beta, cu = s["case"], _beta(s["case"]), s["cu"].tolist()
    told = s["y"] >= 0
    total = []
    for i in range(2 * c["pairs"]):
        part = logp[cu[i]:cu[i + 1]][told[cu[i]:cu[i + 1]]]
        total.append(part.sum() / (max(len(part), 1) if c["mean"] else 1))
    total = torch.stack(total)
    ratio = total if s["ref"] is None else total - s["ref"].double()
    delta = ratio[0::2] - ratio[1::2]
    x = beta * delta - _margin(c)
    pair = {"sigmoid": lambda: -torch.nn.functional.logsigmoid(x), "hinge": lambda: torch.relu(1 - x),
            "ipo": lambda: (delta - 0.5 / beta) ** 2}[c["kind"]]()
    return pair.mean(), dict(loss=pair.mean().detach().reshape(1), pair_loss=pair.detach(), seq_logp=total.detach())
