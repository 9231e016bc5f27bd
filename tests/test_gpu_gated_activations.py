"""GPU checks of the gated block's activations and their slopes over their whole range,
relative to their own size.  One column of x and the weights is set, so that the
projections are exact: g on a grid, u a power of two.

Tolerances.  An activation is a product of a few fp32 factors: 16 roundings of 2^-24,
and an exponential whose argument z is rounded too, which moves it by z 2^-24 a
rounding (at most four); a factor below fp32's smallest normal number 2^-126 may be 0.  The
result is rounded once (2^-8 bf16, 2^-11 fp16).  A slope is a sum of two such terms, each as
exact as that."""
import numpy as np
import pytest
import torch

from oracle import gated as og

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}
E = 2.0 ** -24
NORMAL = 2.0 ** -126


def _exponent(act, g):
    if act == "silu":
        return np.abs(g)
    if act == "gelu":
        return 0.5 * g * g
    return np.abs(2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3))


def _operands(tokens, dtype, u):
    grid = np.arange(-12 * 32, 12 * 32 + 1) / 32.0   # exact in both types
    if dtype == torch.bfloat16:
        grid = torch.from_numpy(grid).to(dtype).double().numpy()
    x, wg, wu = (torch.zeros(n, 8, dtype=dtype) for n in (tokens, grid.size, grid.size))
    x[:, 0], wg[:, 0], wu[:, 0] = 1, torch.from_numpy(grid).to(dtype), u
    return grid, x.cuda(), wg.cuda(), wu.cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("tokens", [1, 40, 200])
def test_values_hold_relative_to_themselves(lib, dtype, act, tokens):
    grid, x, wg, wu = _operands(tokens, dtype, 1024)
    h = lib.gated_forward(x, wg, wu, act).double().cpu().numpy()
    want = 1024 * og.act(act, grid)[0]
    tol = (1.02 * U[dtype] + (16 + 4 * _exponent(act, grid)) * E) * np.abs(want) + 1024 * np.abs(grid) * NORMAL + TINY[dtype]
    err = np.abs(h - want) / tol
    assert np.all(err <= 1), (float(grid[err.max(0).argmax()]), float(err.max()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("tokens", [1, 40])
def test_slopes_hold_relative_to_their_terms(lib, dtype, act, tokens):
    grid, x, wg, wu = _operands(tokens, dtype, 64)
    dh = torch.ones(tokens, grid.size, dtype=dtype, device="cuda")
    _, g, u = lib.gated_forward(x, wg, wu, act, save=True)
    assert np.array_equal(g[0].double().cpu().numpy(), grid) and bool((u == 64).all())
    _, dwg, dwu = lib.gated_backward(x, wg, wu, g, u, dh, act)
    value, slope = og.act(act, grid)
    # value / g, and what is left of the slope
    share = np.where(grid == 0, 0.5, value / np.where(grid == 0, 1, grid))
    terms = np.abs(share) + np.abs(slope - share)
    fp32 = (16 + 4 * _exponent(act, grid)) * E
    un = 1.02 * U[dtype]
    want, got = 64.0 * tokens * slope, dwg[:, 0].double().cpu().numpy()
    lost = (1 + grid * grid) * 2 * NORMAL   # (the second term's factor beside the lost one is at most g (1 + g^2))
    err = np.abs(got - want) / (64.0 * tokens * ((fp32 + un * un) * terms + np.abs(grid) * lost) + un * np.abs(want) + TINY[dtype])
    assert np.all(err <= 1), (float(grid[err.argmax()]), float(err.max()))
    want, got = tokens * value, dwu[:, 0].double().cpu().numpy()
    err = np.abs(got - want) / ((fp32 + un * un + un) * np.abs(want) + tokens * np.abs(grid) * NORMAL + TINY[dtype])
    assert np.all(err <= 1), (float(grid[err.argmax()]), float(err.max()))
