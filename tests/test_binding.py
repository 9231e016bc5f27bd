"""CPU checks of the Python binding's own decisions, with the library's calls replaced."""
import pytest
import torch

import ternary_rank_weight_amd as trw


@pytest.fixture
def forward_calls(monkeypatch):
    """gated_forward by plain products; the list of its calls' `save`."""
    calls = []

    def forward(x, Wg, Wu, act="silu", save=False, **kw):
        calls.append(save)
        g, u = (x @ Wg.t()).detach(), (x @ Wu.t()).detach()
        h = torch.nn.functional.silu(g) * u
        return (h, g, u) if save else h
    monkeypatch.setattr(trw, "gated_forward", forward)
    return calls


def _block():
    gen = torch.Generator().manual_seed(0)
    t = lambda *s: torch.randn(*s, generator=gen)
    return t(3, 8), torch.nn.Parameter(t(5, 8)), torch.nn.Parameter(t(5, 8))


def test_gated_keeps_projections_only_for_a_gradient(forward_calls):
    x, wg, wu = _block()
    with torch.no_grad():
        h = trw.gated(x, wg, wu)
    with torch.inference_mode():
        trw.gated(x, wg, wu)
    trw.gated(x, wg.detach(), wu.detach())
    assert forward_calls == [False] * 3 and not h.requires_grad
    assert trw.gated(x, wg, wu).requires_grad and trw.gated(x.requires_grad_(), wg.detach(), wu.detach()).requires_grad
    assert forward_calls[3:] == [True] * 2


def test_q4_is_read_only():
    # the handle holds addresses: a tensor put in the place of another would leave them to freed memory
    q = trw.Q4.__new__(trw.Q4)
    for name in ("codes", "scales", "mins", "rows", "cols", "group"):
        with pytest.raises(AttributeError):
            setattr(q, name, torch.zeros(4))
        with pytest.raises(AttributeError):
            delattr(q, name)


class _On(torch.Tensor):
    """A host tensor that says it is on CUDA device 1."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 1


def test_workspace_has_to_be_on_the_operands_device():
    ws = torch.zeros(512, dtype=torch.uint8).as_subclass(_On)
    assert trw._scratch(ws, 1) == (ws.data_ptr(), 512)
    assert trw._scratch(None, 0) == (None, 0)
    with pytest.raises(ValueError):
        trw._scratch(ws, 0)
    with pytest.raises(TypeError):
        trw._scratch(torch.zeros(512), 0)
