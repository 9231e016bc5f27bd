"""GPU checks of every form of the linear layer's tiled product, against fp64 on the device.

Tolerances as tests/linear_reference.py derives them, and over a whole output the error that rounding its exact
value leaves, to a tenth: a step of the contraction left out or taken twice moves an output by its own
size over the root of the steps, a hundred times that."""
import numpy as np
import pytest
import torch

from linear_reference import forward_checks, gradient_checks, inputs
from linear_shapes import SHAPES
from oracle import linear as ol

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,cols,rows,act", SHAPES)
def test_form(lib, dtype, tokens, cols, rows, act):
    act = "silu" if act else None
    x, W, b, r, dy = inputs(tokens, cols, rows, dtype, tokens + cols + rows)
    y, z = lib.linear_forward(x, W, b, act, r, save=True)
    assert torch.equal(lib.linear_forward(x, W, b, act, r), y)
    grads = lib.linear_backward(x, W, z, dy, act)
    # dx and dW may be made by one launch: each alone too
    alone = [lib.linear_backward(x, W, z, dy, act, *(i == k for i in range(3)))[k] for k in range(3)]
    assert torch.equal(alone[2], grads[2])
    got = (z, y, *grads, *alone[:2])
    checks = gradient_checks(x, W, b, dy, act)
    for have, (name, want, tol) in zip(got, forward_checks(x, W, b, act, r) + checks + checks[:2]):
        if have is None:
            continue
        err = (have.double() - want).abs()
        assert bool((err <= tol).all()), (name, float((err / tol).max()))
        if have.dtype == dtype:
            assert float(err.norm()) <= 1.1 * float((want.to(dtype).double() - want).norm()), name


def test_reference_is_the_oracle(lib):
    x, W, b, r, dy = inputs(20, 72, 40, torch.float16, 1)
    host = [t.double().cpu().numpy() for t in (x, W, b, r, dy)]
    for act in (None, "silu", "gelu", "gelu_tanh"):
        y, z = ol.forward(*host[:3], act, host[3])
        mine = [v for _, v, _ in forward_checks(x, W, b, act, r) + gradient_checks(x, W, b, dy, act)]
        for a, c in zip(mine, (z, y, *ol.backward(*host[:3], host[4], act))):
            assert np.allclose(a.cpu().numpy(), c, rtol=1e-11, atol=1e-13)
