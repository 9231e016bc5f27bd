"""GPU checks of every form of the gated block's tiled product, against fp64 on the device.

Tolerances as derived in tests/test_gpu_gated_gradients.py, and over a whole output the error
that rounding its exact value leaves, to a tenth: a step of the contraction left out or taken
twice moves an output by its own size over the root of the steps, a hundred times that."""
import pytest
import torch

from gated_reference import E, TINY, U, inputs, references
from gated_shapes import SHAPES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,cols,rows", SHAPES)
def test_form(lib, dtype, tokens, cols, rows):
    x, wg, wu, dh = inputs(tokens, cols, rows, dtype, tokens + cols + rows)
    h, g, u = lib.gated_forward(x, wg, wu, "silu", save=True)
    assert torch.equal(lib.gated_forward(x, wg, wu, "silu"), h)
    X, G, U_ = (t.double() for t in (x, wg, wu))
    for have, W in ((g, G), (u, U_)):
        assert bool(((have.double() - X @ W.t()).abs() <= (cols + 64) * E * (X.abs() @ W.abs().t()) + 1e-30).all())
    gv, uv = X @ G.t(), X @ U_.t()
    want = gv * torch.sigmoid(gv) * uv
    assert float((h.double() - want).norm()) <= 1.1 * float((want.to(dtype).double() - want).norm())
    un, tiny = U[dtype] * 1.02, TINY[dtype]
    for have, (name, want, tol) in zip(lib.gated_backward(x, wg, wu, g, u, dh, "silu"), references(x, wg, wu, dh, "silu")):
        err = (have.double() - want).abs()
        assert bool((err <= tol + un * want.abs() + tiny).all()), (name, float((err / (tol + un * want.abs() + tiny)).max()))
        assert float(err.norm()) <= 1.1 * float((want.to(dtype).double() - want).norm()), name
