"""The LM head's token operators, as a user's program calls them, with their plain forms.

score    log-probabilities of given tokens with the entropy of each position's
         distribution and its K most likely tokens (serving, prompt scoring)
train    log-probabilities and entropies with their gradients (policy and
         preference training on given tokens)
distill  KL divergence from a teacher's top-K logits, loss and gradients

All take hidden states H [N, d] and the head's weight W [V, d] in bf16. Their
values lie on a coarse grid (H on 1/16, W on 1/1024, at most 7 bits and a
sign, as weights and activations held in 8 bits have after widening), so that
every logit is exact in fp32 whatever the order of its sum, and the most likely
tokens are the same ones, ties included (the lowest index first), on each side.
"""
import math

import torch

own = False

IGNORE = -100


def listed():
    return [
        # one decoded token: its log-probability and five alternatives
        dict(name="score_decode_1", op="score", N=1, d=2048, V=151936, K=5, T=1.0),
        # a decoding batch, 20 alternatives at a sampling temperature
        dict(name="score_decode_32", op="score", N=32, d=2048, V=151936, K=20, T=0.7),
        # a few sequences on a wide head with an unpadded vocabulary
        dict(name="score_decode_wide_7", op="score", N=7, d=7168, V=151655, K=10, T=1.0),
        # drafted tokens of a batch verified against the most likely one
        dict(name="score_verify_96", op="score", N=96, d=4096, V=151936, K=1, T=1.0),
        # a small model's batch, latency-bound
        dict(name="score_tiny_256", op="score", N=256, d=256, V=4096, K=8, T=1.0),
        # a prompt scored without alternatives (reference log-probabilities)
        dict(name="score_prompt_1531", op="score", N=1531, d=2048, V=151936, K=0, T=1.0),
        # a packed batch scored with 20 alternatives (a teacher's dump)
        dict(name="score_prompt_8192", op="score", N=8192, d=2048, V=151936, K=20, T=1.0),
        # policy training, small odd sizes
        dict(name="train_odd_250", op="train", N=250, d=264, V=4099, T=0.9),
        # policy training, one micro-batch
        dict(name="train_2048", op="train", N=2048, d=2048, V=151936, T=1.0),
        # a small student
        dict(name="distill_tiny_300", op="distill", N=300, d=256, V=4096, K=16, T=2.0, kind="logits", t="bf16"),
        # one micro-batch of a student, 64 logits kept
        dict(name="distill_2048", op="distill", N=2048, d=2048, V=151936, K=64, T=2.0, kind="logits", t="fp32"),
        # a longer batch on a wider head, the teacher's log-probabilities as they are
        dict(name="distill_5000", op="distill", N=5000, d=4096, V=151936, K=32, T=1.0, kind="logprobs", t="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["score", "score", "train", "distill"])
    most = (8192 * 2048 if op == "score" else 5000 * 4096) * 151936
    while True:
        V = _log(rng, 1000, 151936)
        d = 8 * _log(rng, 256 // 8, 7168 // 8)
        N = _log(rng, 1, 8192) if op == "score" else _log(rng, 64, 5000)
        if N * d * V <= most:
            break
    T = rng.choice([1.0, 1.0, 0.6, 0.85, 1.5, 2.0])
    if op == "score":
        return dict(op=op, N=N, d=d, V=V, K=rng.choice([0, rng.randint(1, 8), rng.randint(9, 64)]), T=T)
    if op == "train":
        return dict(op=op, N=N, d=d, V=V, T=T)
    kind = rng.choice(["logits", "logits", "logprobs"])
    return dict(op=op, N=N, d=d, V=V, K=_log(rng, 1, 128), T=1.0 if kind == "logprobs" else T, kind=kind,
                t=rng.choice(["fp32", "bf16"]))


def _grid(x, steps):
    return (x * steps).round_().clamp_(-127, 127).div_(steps).to(torch.bfloat16)


def prepare(case, seed):
    """Hidden states of a trained model: position i leans towards its token y_i by up to 16 nats."""
    N, d, V, T = case["N"], case["d"], case["V"], case["T"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    sigma = 0.02 if d <= 2048 else 0.015 if d <= 4096 else 0.01
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    W = _grid(randn(V, d).mul_(sigma), 1024.0)
    y = (rand(N).pow(2) * V).long().clamp_(max=V - 1)  # low ids are the frequent ones
    H = randn(N, d).add_(W[y].float() * (16.0 * rand(N, 1) / (sigma * sigma * d)))
    H = _grid(H, 16.0)
    state = dict(case=dict(case), H=H, W=W)
    ignored = rand(N) < 0.05  # padding and prompt positions
    if case["op"] != "distill":
        state["y"] = torch.where(ignored, IGNORE, y) if N > 1 else y
    if case["op"] == "train":
        state["g_logp"] = randn(N) / N              # advantages
        state["g_entropy"] = -0.02 * rand(N) / N    # an entropy bonus
    if case["op"] == "distill":
        K = case["K"]
        k = torch.arange(K, device="cuda")
        stride = 1 + (rand(N, 1) * (V // K - 1)).long()
        idx = (y[:, None] + k * stride) % V         # K different tokens, the position's own first
        t = 8.0 + 12.0 * rand(N, 1) - torch.cumsum(-torch.log1p(-rand(N, K)), 1)
        if case["kind"] == "logprobs":
            t = torch.log_softmax(torch.cat([t, t[:, :1] - 3.0], 1), 1)[:, :K]  # the rest of the vocabulary is one share
        kept = torch.where(rand(N, 1) < 0.2, (rand(N, 1) * K).long() + 1, K)   # some rows keep fewer
        idx = torch.where((k < kept) & ~ignored[:, None], idx, IGNORE)
        state["idx"] = idx.contiguous()
        state["t"] = t.to(torch.bfloat16 if case["t"] == "bf16" else torch.float32).contiguous()
    if case["op"] != "score":
        state["H"].requires_grad_(True)
        state["W"].requires_grad_(True)
    return state


def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own_score(s):
    from chunked_lm_head_linear_gb300 import lce
    c = s["case"]
    logp, _, entropy, top_logp, top_idx = lce.lce_logprobs(s["H"], s["W"], s["y"], top_k=c["K"], temperature=c["T"])
    return dict(logp=logp, entropy=entropy, top_logp=top_logp, top_idx=top_idx)


def _own_train(s):
    from chunked_lm_head_linear_gb300.autograd import FusedLinearLogProbs
    logp, entropy = FusedLinearLogProbs(temperature=s["case"]["T"])(s["H"], s["W"], s["y"])
    dH, dW = torch.autograd.grad([logp, entropy], [s["H"], s["W"]], [s["g_logp"], s["g_entropy"]])
    return dict(logp=logp, entropy=entropy, dH=dH, dW=dW)


def _own_distill(s):
    from chunked_lm_head_linear_gb300.autograd import FusedLinearDistillation
    c = s["case"]
    loss = FusedLinearDistillation(temperature=c["T"], renormalize=c["kind"] == "logits")(s["H"], s["W"], s["idx"], s["t"])
    dH, dW = torch.autograd.grad(loss, [s["H"], s["W"]])
    return dict(loss=loss, dH=dH, dW=dW)


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _head(s):
    """H and W in fp32, the logits over T, their log-sum-exp, softmax and entropy."""
    H, W = s["H"].detach().float(), s["W"].detach().float()
    z = H @ W.t()
    zt = z / s["case"]["T"]
    m = zt.amax(1, keepdim=True)
    e = torch.exp(zt - m)
    total = e.sum(1, keepdim=True)
    entropy = torch.log(total) - (e * (zt - m)).sum(1, keepdim=True) / total
    return H, W, z, zt, m + torch.log(total), e / total, entropy


def _logp(s, zt, lse):
    given = s["y"] != IGNORE
    at = s["y"].clamp(min=0)[:, None]
    return given, at, torch.where(given, (zt.gather(1, at) - lse)[:, 0], 0.0)


def _plain_score(s):
    _, _, z, zt, lse, _, entropy = _head(s)
    _, _, logp = _logp(s, zt, lse)
    K, V = s["case"]["K"], z.shape[1]
    if K == 0:
        return dict(logp=logp, entropy=entropy[:, 0], top_logp=None, top_idx=None)
    bits = (z + 0.0).view(torch.int32).long()       # ordered as the logits are, the lower index first among equals
    keys = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * (1 << 18) + (V - 1 - torch.arange(V, device=z.device))
    idx = V - 1 - (torch.topk(keys, K, dim=1).values & ((1 << 18) - 1))
    return dict(logp=logp, entropy=entropy[:, 0], top_logp=zt.gather(1, idx) - lse, top_idx=idx)


def _plain_train(s):
    H, W, _, zt, lse, p, entropy = _head(s)
    given, at, logp = _logp(s, zt, lse)
    a = torch.where(given, s["g_logp"], 0.0)[:, None]
    G = -p * (a + s["g_entropy"][:, None] * (zt - lse + entropy))
    G.scatter_add_(1, at, a)
    G /= s["case"]["T"]
    return dict(logp=logp, entropy=entropy[:, 0], dH=(G @ W).bfloat16(), dW=(G.t() @ H).bfloat16())


def _plain_distill(s):
    H, W, _, zt, lse, p, _ = _head(s)
    c, kept = s["case"], s["idx"] != IGNORE
    at = s["idx"].clamp(min=0)
    t = torch.where(kept, s["t"].float() / c["T"], -math.inf)
    top = t.amax(1, keepdim=True).clamp(min=-3e38)
    q = torch.exp(t - top) if c["kind"] == "logits" else torch.exp(t)
    q = q / q.sum(1, keepdim=True).clamp(min=1e-38) if c["kind"] == "logits" else q
    n = kept.any(1).sum().clamp(min=1)
    row = torch.where(q > 0, q * (torch.log(q) - zt.gather(1, at) + lse), 0.0).sum(1)
    G = p * q.sum(1, keepdim=True)
    G.scatter_add_(1, at, -q)
    G *= c["T"] / n
    return dict(loss=c["T"] ** 2 * row.sum() / n, dH=(G @ W).bfloat16(), dW=(G.t() @ H).bfloat16())


_own = dict(score=_own_score, train=_own_train, distill=_own_distill)
_plain = dict(score=_plain_score, train=_plain_train, distill=_plain_distill)


def work(case):
    N, d, V = case["N"], case["d"], case["V"]
    rows = 2 * N * d + 2 * V * d + 8 * N                       # H, W and the given tokens
    if case["op"] == "score":
        return dict(bytes=rows + 8 * N + 12 * N * case["K"], flops=2 * N * V * d)
    rows += 2 * N * d + 2 * V * d                              # the gradients
    return dict(bytes=rows + (16 * N if case["op"] == "train" else 12 * N * case["K"]), flops=6 * N * V * d)


def exact(case, seed):
    """The definitions in 64 bits, by blocks of rows; None where the products would take too long."""
    if work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    H, W, T, op = s["H"].detach().double(), s["W"].detach().double(), case["T"], case["op"]
    N = H.shape[0]
    n = int((s["idx"] >= 0).any(1).sum()) if op == "distill" else 0
    got, dH, dW, loss = [], torch.zeros_like(H), torch.zeros_like(W) if op != "score" else None, 0.0
    for r in range(0, N, 512):
        rows = slice(r, min(N, r + 512))
        i = torch.arange(rows.stop - r, device=H.device)
        z = H[rows].matmul(W.t()).div_(T)
        logq = z - torch.logsumexp(z, 1, keepdim=True)         # log-probabilities of every token
        prob = logq.exp()
        if op == "distill":
            q = torch.zeros_like(z)
            idx, t = s["idx"][rows], s["t"][rows].double()
            for j in range(idx.shape[1]):                      # one kept entry a row at a time
                has = idx[:, j] >= 0
                q[i[has], idx[has, j]] = (t[has, j] / T).exp()
            if case["kind"] == "logits":
                q = q / q.sum(1, keepdim=True).clamp(min=1e-300)
            loss += float(torch.special.xlogy(q, q).sum() - (q * logq).sum()) * T * T / max(n, 1)
            grad = (prob * q.sum(1, keepdim=True) - q) * (T / max(n, 1))
        else:
            y = s["y"][rows]
            told = y >= 0
            ent = -(prob * logq).sum(1)
            logp = torch.zeros(len(i), dtype=torch.float64, device=H.device)
            logp[told] = logq[i[told], y[told]]
            got.append((logp, ent, logq.topk(case["K"], dim=1).values if case.get("K") else None))
            if op == "train":
                a = s["g_logp"][rows].double() * told
                e = s["g_entropy"][rows].double()
                grad = -prob * (a[:, None] + e[:, None] * (logq + ent[:, None]))
                grad[i[told], y[told]] += a[told]
                grad /= T
        if op != "score":
            dH[rows] = grad @ W
            dW += grad.t() @ H[rows]
    if op == "distill":
        return dict(loss=torch.tensor(loss, dtype=torch.float64), dH=dH, dW=dW)
    out = dict(logp=torch.cat([x[0] for x in got]), entropy=torch.cat([x[1] for x in got]))
    if op == "train":
        return dict(out, dH=dH, dW=dW)
    return dict(out, top_logp=torch.cat([x[2] for x in got]) if case["K"] else None, top_idx=None)
