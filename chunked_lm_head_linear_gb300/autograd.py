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


class _Distillation(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, W, idx, t, kw):
        need_dH, need_dW = ctx.needs_input_grad[:2]
        if not (need_dH or need_dW):
            loss, _ = lce.lce_distill_forward(H, W, idx, t, **kw)
            return loss.reshape(())
        loss, _, dH, dW = lce.lce_distill_fwd_bwd(H, W, idx, t, dW_dtype=W.dtype, need_dH=need_dH, need_dW=need_dW,
                                                  **kw)
        ctx.grads = dH, dW
        return loss.reshape(())

    def _gradients(ctx, g):
        if ctx.grads is None:
            raise RuntimeError("FusedLinearDistillation: the gradients were handed out by an earlier backward pass "
                               "of this graph; run the forward again")
        dH, dW = ctx.grads
        ctx.grads = None
        lce.lce_scale_grads_bfloat(dH, dW, g)
        return dH, dW, None, None, None

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
