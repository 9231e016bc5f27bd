"""CPU checks of the experts' binding, with the library's calls replaced."""
import pytest
import torch

import ternary_rank_weight_amd as trw


@pytest.fixture
def plain(monkeypatch):
    """Calls on CPU tensors that compute nothing."""
    monkeypatch.setattr(trw, "_op_device", lambda *t: -1)
    monkeypatch.setattr(trw, "_raw_stream", lambda index: 0)
    for name in ("_moe", "_moe_route", "_moe_experts"):
        monkeypatch.setattr(trw, name, lambda *a: 0)


def _operands():
    t = lambda *s: torch.randn(*s).bfloat16()
    return t(4, 16), t(3, 16), t(3, 8, 16), t(3, 8, 16), t(3, 16, 8)


@pytest.mark.parametrize("leaf", range(5))
def test_a_gradient_of_any_result_of_moe_is_refused(plain, leaf):
    ops = [t.requires_grad_(i == leaf) for i, t in enumerate(_operands())]
    y, ids, weights = trw.moe(*ops, 2, routing=True)
    with pytest.raises(RuntimeError, match="has no gradient"):
        y.float().sum().backward()
    # the weights come from x and the router alone
    assert weights.requires_grad == (leaf < 2) and not ids.requires_grad
    if leaf < 2:
        # beside another loss of the same leaf, which has one
        with pytest.raises(RuntimeError, match="has no gradient"):
            (weights.square().sum() + ops[leaf].float().sum()).backward()
    with torch.no_grad():
        assert not any(t.requires_grad for t in trw.moe(*ops, 2, routing=True))


def test_nothing_is_recorded_without_a_leaf(plain):
    assert not any(t.requires_grad for t in trw.moe(*_operands(), 2, routing=True))
