"""The losses' modules where neither the hidden states nor the head need a gradient but another input asks for one, on
fakes of the calls."""
import pytest

from chunked_lm_head_linear_gb300 import lce


@pytest.mark.parametrize("name", ["policy", "preference", "distillation"])
def test_frozen_head_and_inputs_that_ask_for_gradients(monkeypatch, name):
    """advantages, old_logp, ref_logp, weights and a teacher's values get no gradient: with a frozen head the loss is a
    constant, also as a part of a sum with another loss of theirs."""
    torch = pytest.importorskip("torch")
    from chunked_lm_head_linear_gb300 import autograd as A
    monkeypatch.setattr(lce, "lce_policy_forward", lambda H, *a, **kw: (torch.ones(1), torch.zeros(4), torch.zeros(4)))
    monkeypatch.setattr(lce, "lce_preference_forward", lambda H, *a, **kw: (torch.ones(1), torch.zeros(2), torch.zeros(4)))
    monkeypatch.setattr(lce, "lce_distill_forward", lambda H, *a, **kw: (torch.ones(1), torch.zeros(4)))
    H, W, y = torch.zeros(4, 8).bfloat16(), torch.zeros(3, 8).bfloat16(), torch.zeros(4, dtype=torch.int64)
    f = torch.zeros(4, requires_grad=True)
    if name == "policy":
        loss, extra = A.FusedLinearPolicyLoss()(H, W, y, f)
    elif name == "preference":
        loss, extra = A.FusedLinearPreferenceLoss()(H, W, y, torch.arange(5), f)
    else:
        loss, extra = A.FusedLinearDistillation()(H, W, y[:, None], f[:, None]), None
    assert loss.shape == () and not loss.requires_grad and (extra is None or not extra.requires_grad)
    (loss + (f + 1.0).square().sum()).backward()
    assert (f.grad == 2.0).all()
