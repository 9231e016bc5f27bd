"""CPU checks that no operator drops a forward-mode tangent in silence, with the library's calls replaced."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import ternary_rank_weight_amd as trw


@pytest.fixture
def plain(monkeypatch):
    """Calls on CPU tensors that compute nothing."""
    for name, value in (("_op_device", lambda *t: -1), ("_raw_stream", lambda index: 0), ("_current_device", lambda: -1),
                        ("_need", lambda *a: None), ("_linear_scratch", lambda *a: (None, 0, None)),
                        ("_gated_scratch", lambda *a: (None, 0, None)), ("_q4_scratch", lambda *a: (None, 0, None))):
        monkeypatch.setattr(trw, name, value)
    for name in ("_moe", "_moe_route", "_moe_experts", "_linear_forward", "_linear_backward", "_gated_forward", "_gated_backward",
                 "_q4_apply", "_q4_gated"):
        monkeypatch.setattr(trw, name, lambda *a: 0)


def _normal(*shape):
    return torch.randn(*shape).bfloat16()


def _q4():
    return trw.Q4(torch.zeros(256, dtype=torch.int32), torch.zeros(64, dtype=torch.bfloat16), None, 8, 16, 32)


IDS = torch.zeros(4, 2, dtype=torch.int32)
EXPERTS = (3, 8, 16), (3, 8, 16), (3, 16, 8)
# name: (call, shapes of its operands)
CALLS = {
    "linear": (lambda x, W, b, r: trw.linear(x, W, b, "silu", r), ((4, 16), (8, 16), (8,), (4, 8))),
    "linear, x and W": (lambda x, W: trw.linear(x, W), ((4, 16), (8, 16))),
    "linear_forward": (lambda x, W, b, r: trw.linear_forward(x, W, b, None, r), ((4, 16), (8, 16), (8,), (4, 8))),
    "moe": (lambda x, Wr, *w: trw.moe(x, Wr, *w, 2), ((4, 16), (3, 16), *EXPERTS)),
    "moe_route": (lambda x, Wr: trw.moe_route(x, Wr, 2)[1], ((4, 16), (3, 16))),
    "moe_experts": (lambda x, p, *w: trw.moe_experts(x, IDS, p, *w), ((4, 16), (4, 2), *EXPERTS)),
    "gated": (lambda x, Wg, Wu: trw.gated(x, Wg, Wu), ((4, 16), (8, 16), (8, 16))),
    "gated_forward": (lambda x, Wg, Wu: trw.gated_forward(x, Wg, Wu), ((4, 16), (8, 16), (8, 16))),
    "q4_apply": (lambda x: trw.q4_apply(_q4(), x), ((4, 16),)),
    "q4_gated": (lambda x: trw.q4_gated(_q4(), _q4(), x), ((4, 16),)),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_tangent_is_refused(plain, name):
    call, shapes = CALLS[name]
    for k in range(len(shapes)):
        ops = [_normal(*s) for s in shapes]
        with fwd.dual_level():
            call(*ops)   # a level alone changes nothing
            duals = [fwd.make_dual(t, torch.ones_like(t)) if i == k else t for i, t in enumerate(ops)]
            with pytest.raises(RuntimeError, match="forward-mode"):
                call(*duals)
            with torch.no_grad(), pytest.raises(RuntimeError, match="forward-mode"):   # (tangents pass there too)
                call(*duals)
            call(*(t.detach() for t in duals))
        call(*ops)


@pytest.mark.parametrize("name", CALLS)
def test_a_tangent_beside_a_leaf_is_refused(plain, name):
    call, shapes = CALLS[name]
    if len(shapes) < 2:
        return
    ops = [_normal(*s) for s in shapes]
    with fwd.dual_level():
        ops[0] = fwd.make_dual(ops[0], torch.ones_like(ops[0]))
        ops[1].requires_grad_()
        with pytest.raises(RuntimeError):
            call(*ops)


@pytest.mark.parametrize("name", ["linear", "moe", "gated"])
def test_functional_derivatives_are_refused(plain, name):
    call, shapes = CALLS[name]
    ops = [_normal(*s) for s in shapes]
    with pytest.raises(RuntimeError):
        torch.func.jvp(lambda x: call(x, *ops[1:]), (ops[0],), (ops[0],))
