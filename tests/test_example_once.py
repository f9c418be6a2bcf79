"""The example's differentiable operators refuse a second derivative instead of
dropping it (no GPU needed: stand-ins for the library's calls)."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import fast_weight_model as example  # noqa: E402


class Calls:
    embed = staticmethod(lambda ids, table, scale: (scale * table[ids]).detach())
    embed_grad = staticmethod(lambda ids, dy, rows, scale, grad_dtype: torch.zeros(rows, dy.shape[-1]).index_add_(
        0, ids, scale * dy.detach()))
    layer_norm = staticmethod(lambda x, w, b, mean, rstd: x.detach().clone())
    layer_norm_grad = staticmethod(lambda dy, x, w, mean, rstd: (dy.detach().clone(), torch.zeros_like(w), torch.zeros_like(w)))
    delta_rule = staticmethod(lambda q, k, v, g, beta: v.detach().clone())
    delta_rule_grad = staticmethod(lambda q, k, v, g, beta, dy: tuple(
        torch.zeros_like(t) for t in (q, k)) + (dy.detach().clone(), torch.zeros_like(g), torch.zeros_like(beta)))


def tensor(*shape):
    return torch.randn(*shape, requires_grad=True)


CASES = {
    "Embed": lambda: (torch.arange(4), tensor(10, 8), 2.0),
    "LayerNorm": lambda: (tensor(4, 8), tensor(8), tensor(8)),
    "DeltaRule": lambda: (tensor(1, 4, 1, 8), tensor(1, 4, 1, 8), tensor(1, 4, 1, 8), tensor(1, 4, 1), tensor(1, 4, 1)),
}


@pytest.mark.parametrize("name", CASES)
def test_a_second_derivative_is_an_error(monkeypatch, name):
    monkeypatch.setattr(example, "ittt", Calls)
    args = CASES[name]()
    inputs = [a for a in args if isinstance(a, torch.Tensor) and a.requires_grad]
    y = getattr(example, name).apply(*args)
    first = torch.autograd.grad((y ** 2).sum(), inputs, create_graph=True)
    assert any(g.abs().sum() > 0 for g in first)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        sum((g * a).sum() for g, a in zip(first, inputs)).backward()
