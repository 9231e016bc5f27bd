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

from gated_reference import TINY, U, inputs, references
from oracle import gated as og

pytestmark = pytest.mark.gpu


def _gradients(lib, x, wg, wu, dh, act):
    _, g, u = lib.gated_forward(x, wg, wu, act, save=True)
    return lib.gated_backward(x, wg, wu, g, u, dh, act)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,cols,rows", [
    (1, 64, 40), (2, 470, 260), (31, 72, 300), (32, 130, 63), (33, 130, 63), (64, 200, 640), (65, 200, 640),
    (96, 264, 100), (128, 256, 512), (129, 333, 129), (300, 520, 1032), (777, 141, 201), (1024, 512, 384), (5, 33000, 72)])
def test_each_gradient_is_rounded_once(lib, dtype, tokens, cols, rows):
    act = ("silu", "gelu", "gelu_tanh")[(tokens + cols) % 3]
    x, wg, wu, dh = inputs(tokens, cols, rows, dtype, tokens + cols)
    got = _gradients(lib, x, wg, wu, dh, act)
    un, tiny = U[dtype] * 1.02, TINY[dtype]
    for have, (name, want, tol) in zip(got, references(x, wg, wu, dh, act)):
        err = (have.double() - want).abs() / (tol + un * want.abs() + tiny)
        assert bool((err <= 1).all()), (name, float(err.max()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens", [1, 3, 40, 200, 800])
def test_error_is_that_of_rounded_gradients(lib, dtype, tokens):
    # over a whole gradient the error is what rounding its exact value leaves, to a tenth
    x, wg, wu, dh = inputs(tokens, 256, 320, dtype, tokens)
    got = _gradients(lib, x, wg, wu, dh, "silu")
    for have, (name, want, _) in zip(got, references(x, wg, wu, dh, "silu")):
        rounded = float((want.to(dtype).double() - want).norm())
        assert float((have.double() - want).norm()) <= 1.1 * rounded, name


def _scaled(tokens, cols, rows, x, wg, wu, dh, seed):
    """fp16 operands of the given standard deviations."""
    rng = np.random.default_rng(seed)
    t = lambda s, *shape: torch.from_numpy((s * rng.standard_normal(shape)).astype(np.float32)).half().cuda()
    return t(x, tokens, cols), t(wg, rows, cols), t(wu, rows, cols), t(dh, tokens, rows)


def _check_fp16_range(lib, ops, names, large):
    x, wg, wu, dh = ops
    X, G, U_, D = (t.double() for t in ops)
    gv, uv = X @ G.t(), X @ U_.t()
    a, slope = (torch.from_numpy(t).cuda() for t in og.act("silu", gv.cpu().numpy()))
    top = max(float((D * uv * slope).abs().max()), float((D * a).abs().max()))
    assert (top > 2e5) if large else (top < 1e-4)
    got = _gradients(lib, x, wg, wu, dh, "silu")
    # the smaller part holds steps of 2^-24 where the largest value is brought to 2^14 or more
    refs = references(x, wg, wu, dh, "silu", step=2.0 ** -39 * top)
    for have, (name, want, tol) in zip(got, refs):
        if name not in names:
            continue
        assert float(want.abs().max()) < 60000 and float(want.abs().max()) > 2.0 ** -12
        err = (have.double() - want).abs() / (tol + 1.02 * 2.0 ** -11 * want.abs() + 2.0 ** -25)
        assert bool((err <= 1).all()), (name, float(err.max()))


@pytest.mark.parametrize("tokens,cols,rows", [(1, 256, 32), (9, 256, 32), (70, 251, 31), (300, 256, 32)])
def test_fp16_gradients_in_range_from_larger_dg_and_du(lib, tokens, cols, rows):
    # dg and du pass 65504 (dh of 5000 times projections of 32), dx or dWg and dWu do not
    _check_fp16_range(lib, _scaled(tokens, cols, rows, 400, 0.005, 0.005, 5000, tokens), ("dx",), True)
    _check_fp16_range(lib, _scaled(tokens, cols, rows, 0.002, 1000, 1000, 5000, tokens), ("dWg", "dWu"), True)


@pytest.mark.parametrize("tokens,cols,rows", [(2, 256, 1000), (70, 256, 1000), (900, 251, 65)])
def test_fp16_gradients_from_small_dg_and_du(lib, tokens, cols, rows):
    # dg and du of 1e-6, in fp16 a dozen steps, add up to gradients with all their bits
    _check_fp16_range(lib, _scaled(tokens, cols, rows, 0.002, 30, 30, 1e-6, tokens), ("dx",), False)
    _check_fp16_range(lib, _scaled(tokens, cols, rows, 900, 7e-5, 7e-5, 1e-6, tokens), ("dWg", "dWu"), False)


@pytest.mark.parametrize("tokens", [8, 150])
def test_fp16_large_token_or_unit_leaves_the_others_bits(lib, tokens):
    # one token's dh is 2^30 times the others': their rows of dx keep their values bit for bit
    x, wg, wu, dh = _scaled(tokens, 128, 96, 1, 0.05, 0.05, 2.0 ** -16, tokens)
    _, g, u = lib.gated_forward(x, wg, wu, save=True)
    dx, dwg, dwu = lib.gated_backward(x, wg, wu, g, u, dh)
    loud = dh.clone()
    loud[3] = (dh[3].float().sign() * 2.0 ** 14).half()
    other = lib.gated_backward(x, wg, wu, g, u, loud)[0]
    keep = [t for t in range(tokens) if t != 3]
    assert torch.equal(other[keep], dx[keep]) and not torch.equal(other[3], dx[3])
    # and one hidden unit's: the others' rows of dWg and dWu
    loud = dh.clone()
    loud[:, 5] = (dh[:, 5].float().sign() * 2.0 ** 14).half()
    other = lib.gated_backward(x, wg, wu, g, u, loud)
    keep = [f for f in range(96) if f != 5]
    assert torch.equal(other[1][keep], dwg[keep]) and torch.equal(other[2][keep], dwu[keep])


@pytest.mark.parametrize("tokens", [5, 100])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_bad_token_stays_in_its_row_of_dx(lib, dtype, tokens):
    x, wg, wu, dh = inputs(tokens, 72, 136, dtype, 6)
    _, g, u = lib.gated_forward(x, wg, wu, save=True)
    dx = lib.gated_backward(x, wg, wu, g, u, dh)[0]
    bad = dh.clone()
    bad[2, 9], bad[4, 0] = float("nan"), float("inf")
    got, dwg, _ = lib.gated_backward(x, wg, wu, g, u, bad)
    keep = [t for t in range(tokens) if t not in (2, 4)]
    assert torch.equal(got[keep], dx[keep])
    assert bool(torch.isnan(got[2]).all()) and not bool(torch.isfinite(got[4]).any())
    assert bool(torch.isnan(dwg[9]).all()) and bool(torch.isfinite(dwg[[f for f in range(136) if f not in (0, 9)]]).all())


@pytest.mark.parametrize("tokens,cols,rows", [(2, 136, 72), (70, 136, 72), (150, 203, 65)])
def test_fp16_scales_in_a_used_workspace_and_in_a_graph(lib, tokens, cols, rows):
    # the largest magnitudes of the call before, in the workspace, do not reach the next
    x, wg, wu, dh = inputs(tokens, cols, rows, torch.float16, 3)
    _, g, u = lib.gated_forward(x, wg, wu, save=True)
    want = lib.gated_backward(x, wg, wu, g, u, dh)
    need = lib.gated_backward_workspace_bytes(tokens, cols, rows, cols % 8 == 0)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    lib.gated_backward(x, wg, wu, g, u, dh * 1000, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(lib.gated_backward(x, wg, wu, g, u, dh, workspace=ws), want))
    static = dh.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = lib.gated_backward(x, wg, wu, g, u, static, workspace=ws)
    for k in (1000, 0.01, 1, 30):
        static.copy_(dh * k)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, lib.gated_backward(x, wg, wu, g, u, dh * k)))
