"""GPU checks of the gated block's gradients: dg and du enter the products with more
bits than the operands' type has, at every token count, and each gradient is then
rounded once.  References in fp64 on the device.

Tolerances.  The kept projections are off by at most (cols + 64) 2^-24 of their terms'
magnitude, and activation values and slopes carry a few fp32 roundings of their own.
dg and du are held in two 16-bit parts: the first is off by u = half an ulp (2^-8
bf16, 2^-11 fp16), the second by u of that.  A sum of n terms of total magnitude S in
fp32 is off by at most (n + 64) 2^-24 S, and each gradient is rounded once by u; fp16 adds
its subnormal step."""
import numpy as np
import pytest
import torch

from oracle import gated as og

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}
E = 2.0 ** -24


def _inputs(tokens, cols, rows, dtype, seed):
    rng = np.random.default_rng(seed)
    t = lambda a: torch.from_numpy(a.astype(np.float32)).to(dtype).cuda()
    scale = 1.0 / np.sqrt(cols)
    return (t(rng.standard_normal((tokens, cols))), t(scale * 1.5 * rng.standard_normal((rows, cols))),
            t(scale * rng.standard_normal((rows, cols))), t(rng.standard_normal((tokens, rows))))


def _references(x, wg, wu, dh, act, step=None):
    """[(name, fp64 gradient, tolerance before the output's rounding)].  step: the smallest difference of
    two dg or du that the parts hold (the subnormal step of dh's type by default)."""
    dtype, cols, tokens, rows = x.dtype, x.shape[1], x.shape[0], wg.shape[0]
    X, G, U_, D = (t.double() for t in (x, wg, wu, dh))
    gv, uv = X @ G.t(), X @ U_.t()
    a, slope = (torch.from_numpy(t).cuda() for t in og.act(act, gv.cpu().numpy()))
    eg, eu = (cols + 64) * E * (X.abs() @ G.abs().t()), (cols + 64) * E * (X.abs() @ U_.abs().t())
    ea, es = 1.13 * eg + 16 * E * gv.abs(), 0.9 * eg + 32 * E * (1 + gv.abs())
    un = U[dtype] * 1.02
    dg, du = D * uv * slope, D * a
    if step is None:
        step = TINY[dtype]
    edg = D.abs() * ((uv.abs() + eu) * es + eu * slope.abs()) + un ** 2 * dg.abs() + step
    edu = D.abs() * ea + un ** 2 * du.abs() + step
    mg, mu = dg.abs() + edg, du.abs() + edu
    return [("dx", dg @ G + du @ U_, edg @ G.abs() + edu @ U_.abs() + (4 * rows + 128) * E * (mg @ G.abs() + mu @ U_.abs())),
            ("dWg", dg.t() @ X, edg.t() @ X.abs() + (2 * tokens + 64) * E * (mg.t() @ X.abs())),
            ("dWu", du.t() @ X, edu.t() @ X.abs() + (2 * tokens + 64) * E * (mu.t() @ X.abs()))]


def _gradients(lib, x, wg, wu, dh, act):
    _, g, u = lib.gated_forward(x, wg, wu, act, save=True)
    return lib.gated_backward(x, wg, wu, g, u, dh, act)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,cols,rows", [
    (1, 64, 40), (2, 470, 260), (31, 72, 300), (32, 130, 63), (33, 130, 63), (64, 200, 640), (65, 200, 640),
    (96, 264, 100), (128, 256, 512), (129, 333, 129), (300, 520, 1032), (777, 141, 201), (1024, 512, 384), (5, 33000, 72)])
def test_each_gradient_is_rounded_once(lib, dtype, tokens, cols, rows):
    act = ("silu", "gelu", "gelu_tanh")[(tokens + cols) % 3]
    x, wg, wu, dh = _inputs(tokens, cols, rows, dtype, tokens + cols)
    got = _gradients(lib, x, wg, wu, dh, act)
    un, tiny = U[dtype] * 1.02, TINY[dtype]
    for have, (name, want, tol) in zip(got, _references(x, wg, wu, dh, act)):
        err = (have.double() - want).abs() / (tol + un * want.abs() + tiny)
        assert bool((err <= 1).all()), (name, float(err.max()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens", [1, 3, 40, 200, 800])
def test_error_is_that_of_rounded_gradients(lib, dtype, tokens):
    # over a whole gradient the error is what rounding its exact value leaves, to a tenth
    x, wg, wu, dh = _inputs(tokens, 256, 320, dtype, tokens)
    got = _gradients(lib, x, wg, wu, dh, "silu")
    for have, (name, want, _) in zip(got, _references(x, wg, wu, dh, "silu")):
        rounded = float((want.to(dtype).double() - want).norm())
        assert float((have.double() - want).norm()) <= 1.1 * rounded, name
