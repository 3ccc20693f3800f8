"""PyTorch autograd wrapper of the fused LM-head linear + cross-entropy.

    loss_fn = FusedLinearCrossEntropy(ignore_index=-100)
    loss = loss_fn(H, W, y)      # H [N, d] bf16, W [V, d] bf16, y [N] int64, all on the GPU
    loss.backward()              # H.grad, W.grad (in W's dtype: autograd casts the fp32 dW to it)

The forward pass runs the whole fused forward + backward (lce_fwd_bwd with an
upstream gradient of 1) and keeps dH and dW; the backward pass scales them by
the actual upstream gradient with lce_scale_grads (a device-side no-op when it
is 1). This is the arrangement of the fused loss on "XTuner on Ascend 910C:
Qwen3.5-2B training optimisation" (section 3.1.4: one fused kernel produces
d_input and d_weight, no d_logits is kept), and it costs 6 N V d flops.
``recompute=True`` instead saves only lse in the forward and recomputes the
logits in the backward (lce_backward, 8 N V d flops) -- for when the
gradients should not be held between the passes.

The library's dW is fp32; autograd hands a leaf its gradient in the leaf's own
dtype, so a bf16 W receives bf16 gradients. Callers that keep fp32 weight
gradients (gradient accumulation over micro-batches, fp32 reduction across
ranks) call ``lce.lce_fwd_bwd`` with their fp32 buffer as ``dW`` and
``accumulate_dW=True`` instead.

FusedLinearLogProbs and FusedLinearDistillation wrap the token operators
(lce_logprobs_keep, lce_distill_fwd_bwd) the same way: log-probabilities and
entropies of given tokens, whose upstream gradients are known only in the
backward, save logp, entropy and the rows' statistics, and the logits of a
batch of one chunk (else they are recomputed there); the distillation loss
computes its gradients in the forward and scales them in the backward.
FusedLinearPolicyLoss and FusedLinearPreferenceLoss wrap lce_policy_fwd_bwd and
lce_preference_fwd_bwd as the distillation loss is wrapped. FusedLayerNorm is
the norm in front of any of them (lce_layernorm_forward / _backward).
Gradients nobody needs (a frozen W, torch.no_grad) are not computed, and nothing
is kept for them.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import lce


class _FusedLCE(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, W, y, opts):
        loss, _, dH, dW = lce.lce_fwd_bwd(H, W, y, **opts)
        ctx.save_for_backward(dH, dW)
        return loss.reshape(())

    @staticmethod
    def backward(ctx, g):
        dH, dW = ctx.saved_tensors
        g = g.reshape(1).to(torch.float32).contiguous()
        lce.lce_scale_grads(dH, dW, g)
        return dH, dW, None, None


class _RecomputeLCE(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, W, y, opts):
        loss, lse = lce.lce_forward(H, W, y, **opts)
        ctx.save_for_backward(H, W, y, lse)
        ctx.opts = opts
        return loss.reshape(())

    @staticmethod
    def backward(ctx, g):
        H, W, y, lse = ctx.saved_tensors
        g = g.reshape(1).to(torch.float32).contiguous()
        dH, dW = lce.lce_backward(H, W, y, lse, g, **ctx.opts)
        return dH, dW, None, None


class FusedLinearCrossEntropy(torch.nn.Module):
    """Token-level cross-entropy of the LM-head logits H W^T (mean over tokens
    whose label is not ignore_index), fused and chunked on the GPU."""

    def __init__(self, ignore_index: int = -100, reduction: str = "mean", chunk_tokens=0, recompute: bool = False):
        super().__init__()
        self.opts = dict(ignore_index=ignore_index, reduction=reduction, chunk_tokens=chunk_tokens)
        self.recompute = recompute

    def forward(self, H, W, y):
        fn = _RecomputeLCE if self.recompute else _FusedLCE
        return fn.apply(H, W, y, self.opts)


def _first_order(gradients):
    """A Function's backward whose gradients are not differentiable themselves:
    once_differentiable, whose bookkeeping is left out where no graph of the
    backward is asked for."""
    checked = once_differentiable(gradients)

    def backward(ctx, *g):
        return checked(ctx, *g) if torch.is_grad_enabled() else gradients(ctx, *g)

    return staticmethod(backward)


class _LogProbs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, W, y, temperature, keep, opts):
        logits = None
        if keep and (ctx.needs_input_grad[0] or ctx.needs_input_grad[1]):
            logits = torch.empty((H.shape[0], (W.shape[0] + 255) // 256 * 256), dtype=torch.float32, device=H.device)
        logp, _, entropy, _, _, stats = lce.lce_logprobs_keep(H, W, y, temperature=temperature, logits=logits, **opts)
        ctx.save_for_backward(H, W, y, logp, entropy, stats, logits)
        ctx.temperature, ctx.opts = temperature, opts
        ctx.set_materialize_grads(False)   # an output nobody used comes back as None
        return logp, entropy

    def _gradients(ctx, g_logp, g_entropy):
        H, W, y, logp, entropy, stats, logits = ctx.saved_tensors
        g_logp = torch.zeros_like(logp) if g_logp is None else g_logp.contiguous()
        g_entropy = None if g_entropy is None else g_entropy.contiguous()
        # the forward checked its tensors, autograd that the gradients are like the outputs
        need_dH, need_dW = ctx.needs_input_grad[:2]
        dH, dW = lce._logprobs_backward(H, W, y, logp, None, stats, entropy, g_logp, g_entropy, logits, ctx.temperature,
                                        lce.LCE_DW_BF16, None, need_dH, need_dW, None, None, ctx.opts)
        return dH, dW, None, None, None, None

    backward = _first_order(_gradients)


class FusedLinearLogProbs(torch.nn.Module):
    """logp [N] of the tokens y and entropy [N] of softmax(H W^T / temperature),
    both differentiable in H and W (fp32; logp is 0 where y is ignore_index).

    ``recompute``: True: the backward recomputes the logits (8 N V d flops in
    all); False: the forward keeps them for it (4 N V bytes, 6 N V d flops);
    None: they are kept when the batch is one chunk (chunk_tokens, or fewer than
    6144 tokens), so that the memory held stays O(chunk V), and d is at least
    1536: below, reading them costs more than the product, or as much. Forward and
    backward at V = 151936, microseconds recomputed and kept:

        rows        512           1024          2048          4096
        d =  768    398 /  471    659 /  726    1235 / 1344   2492 /  2601
        d = 1024    482 /  536    799 /  847    1570 / 1592   3081 /  3070
        d = 1536    724 /  741   1150 / 1095    2205 / 2047   4475 /  4205
        d = 2048    952 /  918   1515 / 1379    2944 / 2602   6011 /  5336
        d = 4096   1779 / 1531   3129 / 2598    6101 / 4962  12359 / 10055

    (128 rows: kept is ahead from d = 1024 on, 338 / 318, with 78 MB of logits.)"""

    def __init__(self, temperature: float = 1.0, ignore_index: int = -100, chunk_tokens=0, recompute=None):
        super().__init__()
        self.temperature = temperature
        self.recompute = recompute
        self.opts = dict(ignore_index=ignore_index, chunk_tokens=chunk_tokens)

    def forward(self, H, W, y):
        if not torch.is_grad_enabled():   # inside a Function grad mode is always off: only here it is the caller's
            logp, _, entropy, _, _ = lce.lce_logprobs(H, W, y, temperature=self.temperature, **self.opts)
            return logp, entropy
        keep = not self.recompute
        if self.recompute is None:
            chunk = self.opts["chunk_tokens"]
            keep = chunk != "auto" and H.shape[0] <= (chunk or 6143) and H.shape[1] >= 1536
        return _LogProbs.apply(H, W, y, self.temperature, keep, self.opts)


def _scaled(ctx, g, what):
    """The gradients that the forward computed, times the upstream one; handed out once, as they are scaled in place."""
    if ctx.grads is None:
        raise RuntimeError(f"{what}: the gradients were handed out by an earlier backward pass of this graph; run the "
                           "forward again")
    dH, dW = ctx.grads
    ctx.grads = None
    lce.lce_scale_grads_bfloat(dH, dW, g)
    return dH, dW


class _Distillation(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, W, idx, t, kw):
        need_dH, need_dW = ctx.needs_input_grad[:2]
        if not (need_dH or need_dW):
            loss = lce.lce_distill_forward(H, W, idx, t, **kw)[0].reshape(())
            ctx.mark_non_differentiable(loss)   # an input without a gradient here (t) may ask for one
            return loss
        loss, _, dH, dW = lce.lce_distill_fwd_bwd(H, W, idx, t, dW_dtype=W.dtype, need_dH=need_dH, need_dW=need_dW,
                                                  **kw)
        ctx.grads = dH, dW
        return loss.reshape(())

    def _gradients(ctx, g):
        return *_scaled(ctx, g, "FusedLinearDistillation"), None, None, None

    backward = _first_order(_gradients)


class FusedLinearDistillation(torch.nn.Module):
    """KL divergence of softmax(H W^T / temperature) from a teacher's top tokens
    idx [N, K] with values t [N, K], times temperature^2, mean over the rows that
    keep an entry (lce.lce_distill_fwd_bwd). Its gradients are computed in the
    forward pass in bf16 and scaled by the upstream gradient in the backward,
    where they are rounded once more unless it is a power of two (a weight given
    to lce.lce_distill_fwd_bwd as grad_loss is in their one rounding). The
    teacher's values get no gradient."""

    def __init__(self, temperature: float = 1.0, renormalize: bool = True, ignore_index: int = -100,
                 reduction: str = "mean", chunk_tokens=0):
        super().__init__()
        self.kw = dict(temperature=temperature, renormalize=renormalize, ignore_index=ignore_index,
                       reduction=reduction, chunk_tokens=chunk_tokens)

    def forward(self, H, W, idx, t):
        if not torch.is_grad_enabled():
            return lce.lce_distill_forward(H, W, idx, t, **self.kw)[0].reshape(())
        return _Distillation.apply(H, W, idx, t, self.kw)


class _PolicyLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, W, y, advantages, old_logp, ref_logp, weights, kw):
        need_dH, need_dW = ctx.needs_input_grad[:2]
        if not (need_dH or need_dW):
            loss, logp, _ = lce.lce_policy_forward(H, W, y, advantages, old_logp, ref_logp, weights=weights, **kw)
            loss = loss.reshape(())
            ctx.mark_non_differentiable(loss, logp)   # advantages, old_logp, ref_logp or weights may ask for a gradient
            return loss, logp
        loss, logp, _, dH, dW = lce.lce_policy_fwd_bwd(H, W, y, advantages, old_logp, ref_logp, weights=weights,
                                                       dW_dtype=W.dtype, need_dH=need_dH, need_dW=need_dW, **kw)
        ctx.grads = dH, dW
        ctx.mark_non_differentiable(logp)
        return loss.reshape(()), logp

    def _gradients(ctx, g, _):
        return *_scaled(ctx, g, "FusedLinearPolicyLoss"), None, None, None, None, None, None

    backward = _first_order(_gradients)


class FusedLinearPolicyLoss(torch.nn.Module):
    """The clipped policy loss with a KL term (lce.lce_policy_fwd_bwd) of the tokens
    y [N] under softmax(H W^T / temperature), and their log-probabilities logp
    [N] (without a gradient: for ratios and KL divergences to look at). The
    gradients are computed in the forward pass in bf16 and scaled by the
    upstream gradient in the backward, where they are rounded once more unless
    it is a power of two. advantages, old_logp, ref_logp and weights (fp32 [N])
    get no gradient."""

    def __init__(self, temperature: float = 1.0, clip_low: float = 0.2, clip_high: float = 0.2, dual_clip: float = 0.0,
                 kl: str = "none", kl_coef: float = 0.0, ignore_index: int = -100, reduction: str = "mean",
                 chunk_tokens=0):
        super().__init__()
        self.kw = dict(temperature=temperature, clip_low=clip_low, clip_high=clip_high, dual_clip=dual_clip, kl=kl,
                       kl_coef=kl_coef, ignore_index=ignore_index, reduction=reduction, chunk_tokens=chunk_tokens)

    def forward(self, H, W, y, advantages, old_logp=None, ref_logp=None, weights=None):
        if not torch.is_grad_enabled():
            loss, logp, _ = lce.lce_policy_forward(H, W, y, advantages, old_logp, ref_logp, weights=weights, **self.kw)
            return loss.reshape(()), logp
        return _PolicyLoss.apply(H, W, y, advantages, old_logp, ref_logp, weights, self.kw)


class _PreferenceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, W, y, cu_seqlens, ref_logp, kw):
        need_dH, need_dW = ctx.needs_input_grad[:2]
        if not (need_dH or need_dW):
            loss, _, seq_logp = lce.lce_preference_forward(H, W, y, cu_seqlens, ref_logp, **kw)
            loss = loss.reshape(())
            ctx.mark_non_differentiable(loss, seq_logp)   # ref_logp may ask for a gradient
            return loss, seq_logp
        loss, _, seq_logp, dH, dW = lce.lce_preference_fwd_bwd(H, W, y, cu_seqlens, ref_logp, dW_dtype=W.dtype,
                                                               need_dH=need_dH, need_dW=need_dW, **kw)
        ctx.grads = dH, dW
        ctx.mark_non_differentiable(seq_logp)
        return loss.reshape(()), seq_logp

    def _gradients(ctx, g, _):
        return *_scaled(ctx, g, "FusedLinearPreferenceLoss"), None, None, None, None

    backward = _first_order(_gradients)


class FusedLinearPreferenceLoss(torch.nn.Module):
    """The loss of paired sequences' log ratios (lce.lce_preference_fwd_bwd), and the
    sequences' log-probabilities seq_logp [2 P] (without a gradient: times beta,
    less the reference's, they are the rewards). cu_seqlens [2 P + 1] bounds
    chosen and rejected sequences in turn. The gradients are computed in the
    forward pass, as FusedLinearPolicyLoss's."""

    def __init__(self, kind: str = "sigmoid", beta: float = 0.1, label_smoothing: float = 0.0, margin: float = 0.0,
                 average: bool = False, temperature: float = 1.0, ignore_index: int = -100, reduction: str = "mean",
                 chunk_tokens=0):
        super().__init__()
        self.kw = dict(kind=kind, beta=beta, label_smoothing=label_smoothing, margin=margin, average=average,
                       temperature=temperature, ignore_index=ignore_index, reduction=reduction,
                       chunk_tokens=chunk_tokens)

    def forward(self, H, W, y, cu_seqlens, ref_logp=None):
        if not torch.is_grad_enabled():
            loss, _, seq_logp = lce.lce_preference_forward(H, W, y, cu_seqlens, ref_logp, **self.kw)
            return loss.reshape(()), seq_logp
        return _PreferenceLoss.apply(H, W, y, cu_seqlens, ref_logp, self.kw)


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b, eps):
        H, mean, rstd = lce.lce_layernorm_forward(x, w, b, eps)
        ctx.save_for_backward(x, w, mean, rstd)
        ctx.bias = None if b is None else b.dtype
        return H

    def _gradients(ctx, dH):
        x, w, mean, rstd = ctx.saved_tensors
        need_dx, need_dw, need_db = ctx.needs_input_grad[:3]
        dx, dw, db = lce.lce_layernorm_backward(x, w, mean, rstd, dH.contiguous(), bias=need_db, need_dx=need_dx,
                                                need_dw=need_dw)
        return dx, None if dw is None else dw.to(w.dtype), None if db is None else db.to(ctx.bias), None

    backward = _first_order(_gradients)


class FusedLayerNorm(torch.nn.Module):
    """Layer norm in front of the head: H (bf16 [N, d]) of x (bf16 or fp32 [N, d]) with
    weight w and bias b (fp32 or bf16 [d], or None), differentiable in all three
    (lce.lce_layernorm_forward / lce_layernorm_backward)."""

    def __init__(self, eps: float = 1e-5):
        super().__init__()
        self.eps = eps

    def forward(self, x, w=None, b=None):
        if not torch.is_grad_enabled():
            return lce.lce_layernorm_forward(x, w, b, self.eps)[0]
        return _LayerNorm.apply(x, w, b, self.eps)
