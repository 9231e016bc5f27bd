"""GPU checks of every form of the experts' products, against oracle/moe.py in fp64 with the tolerances that
tests/test_gpu_moe.py derives, and over the whole output the error that rounding its exact value leaves, to a tenth: a row, a
part or a stretch of 64 columns left out or taken twice moves outputs by far more."""
import numpy as np
import pytest
import torch

from moe_shapes import SHAPES
from oracle import moe as om
from test_gpu_moe import _check, _host, _inputs

pytestmark = pytest.mark.gpu


def _starting(t, first):
    """t, `first` entries past a multiple of 16 bytes, among values that are not numbers."""
    buf = torch.full((first + t.numel() + 8,), float("nan"), dtype=t.dtype, device="cuda")
    v = buf[first:first + t.numel()].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,cols,rows,experts,top,alike", SHAPES)
def test_form(lib, dtype, tokens, cols, rows, experts, top, alike):
    x, Wr, Wg, Wu, Wd = _inputs(tokens, cols, rows, experts, dtype, tokens + cols + rows)
    if not alike:
        Wg, Wu = _starting(Wg, 1), _starting(Wu, 4)
        assert (Wg.data_ptr() ^ Wu.data_ptr()) & 15
    act = ("silu", "gelu", "gelu_tanh")[(cols + rows) % 3]
    y, ids, weights = _check(lib, (x, Wr, Wg, Wu, Wd), top, act)
    want = om.experts(_host(x), ids.cpu().numpy(), _host(weights), _host(Wg), _host(Wu), _host(Wd), act)
    rounded = torch.from_numpy(want).to(dtype).double().numpy()
    assert np.linalg.norm(_host(y) - want) <= 1.1 * np.linalg.norm(rounded - want)
