"""CPU checks of the linear layer's binding, with the library's calls replaced."""
import pytest
import torch

import ternary_rank_weight_amd as trw


@pytest.fixture
def forward_calls(monkeypatch):
    """linear_forward by a plain product; the list of its calls' `save`."""
    calls = []

    def forward(x, W, bias=None, act=None, residual=None, save=False, **kw):
        calls.append(save)
        z = (x @ W.t() + bias).detach()
        y = torch.nn.functional.silu(z) + residual.detach()
        return (y, z) if save else y
    monkeypatch.setattr(trw, "linear_forward", forward)
    return calls


def _layer():
    gen = torch.Generator().manual_seed(0)
    t = lambda *s: torch.randn(*s, generator=gen)
    return t(3, 8), t(5, 8), t(5), t(3, 5)


def test_keeps_z_only_for_a_gradient_that_needs_it(forward_calls):
    x, W, b, r = _layer()
    leaf = torch.nn.Parameter(W)
    with torch.no_grad():
        assert not trw.linear(x, leaf, b, "silu", r).requires_grad
    with torch.inference_mode():
        trw.linear(x, leaf, b, "silu", r)
    trw.linear(x, W, b, "silu", r)
    dy = torch.randn(3, 5)
    r.requires_grad_()
    trw.linear(x, W, b, "silu", r).backward(dy)   # the residual's gradient is dy
    assert forward_calls == [False] * 4 and torch.equal(r.grad, dy)
    for k in range(3):
        ops = [t.detach().clone().requires_grad_(i == k) for i, t in enumerate((x, W, b))]
        assert trw.linear(*ops, "silu", r.detach()).requires_grad
    assert forward_calls[4:] == [True] * 3
