"""BalanceLoss under autograd: a second derivative, which it does not have, is an error (no GPU: the loss itself is
replaced by a plain one)."""
import pytest
import torch


@pytest.fixture
def b(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    import expert_slot_cache_gb300.binding as b

    def plain(logits, ids, coef, seq_start=None, token_mask=None, sigmoid=False, with_loss=True, with_grad=False, grad_loss=None):
        g = 1.0 if grad_loss is None else grad_loss
        return b.Balance((logits.detach() ** 2).sum() * coef, torch.zeros(1, logits.shape[1], dtype=torch.int32),
                         2 * coef * g * logits.detach() if with_grad else None)

    monkeypatch.setattr(b, "balance_loss", plain)
    return b


def test_second_derivatives_are_refused(b):
    leaf = torch.randn(5, 8, requires_grad=True)
    loss, counts = b.BalanceLoss.apply(leaf, torch.zeros(5, 2, dtype=torch.int32), 0.5)
    (g,) = torch.autograd.grad(loss * 3.0, leaf, create_graph=True)
    assert torch.allclose(g, 3 * leaf.detach())
    with pytest.raises(RuntimeError, match="second derivative"):
        (loss + (g * g).sum()).backward()
    assert not counts.requires_grad


def test_first_derivatives_with_a_graph(b):
    """A graph of the first derivative may be asked for on behalf of other terms."""
    leaf = torch.randn(5, 8, requires_grad=True)
    loss, _ = b.BalanceLoss.apply(leaf, torch.zeros(5, 2, dtype=torch.int32), 0.5)
    other = torch.randn(3, requires_grad=True)
    g, h = torch.autograd.grad(loss * 2.0 + (other ** 3).sum(), (leaf, other), create_graph=True)
    h.sum().backward()
    assert torch.allclose(g.detach(), 2 * leaf.detach()) and torch.allclose(other.grad, 6 * other.detach())
