"""GPU checks of the linear layer, forward and backward, against the formulas in fp64 with the bounds that
tests/linear_reference.py derives, and against differences."""
import pytest
import torch

from linear_reference import U, forward_checks, gradient_checks, inputs

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
ACTS = (None, "silu", "gelu", "gelu_tanh")


def _within(got, checks):
    for have, (name, want, tol) in zip(got, checks):
        if have is None:
            continue
        err = (have.double().view(want.shape) - want).abs()
        assert bool((err <= tol).all()), (name, float((err / tol).max()))


def _check(lib, x, W, bias, residual, dy, act):
    y, z = lib.linear_forward(x, W, bias, act, residual, save=True)
    assert (z is None) == (act is None) and torch.equal(lib.linear_forward(x, W, bias, act, residual), y)
    _within((z, y), forward_checks(x, W, bias, act, residual))
    grads = lib.linear_backward(x, W, z, dy, act)
    _within(grads, gradient_checks(x, W, bias, dy, act))
    return (y, *grads)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("tokens,cols,rows", [
    (1, 1, 1), (1, 64, 128), (3, 8, 16), (2, 7, 5), (16, 128, 64), (17, 72, 40), (33, 200, 136), (64, 256, 512),
    (65, 333, 129), (100, 1000, 24), (130, 63, 65), (257, 264, 300), (300, 520, 1032), (600, 77, 131)])
def test_layer(lib, dtype, tokens, cols, rows):
    for k, act in enumerate(ACTS):
        x, W, b, r, dy = inputs(tokens, cols, rows, dtype, tokens + cols + k, bias=k != 1, residual=k != 2)
        _check(lib, x, W, b, r, dy, act)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True)])
def test_parts_of_the_epilogue(lib, act, bias, residual):
    for tokens in (5, 40, 300):
        _check(lib, *inputs(tokens, 96, 80, BF16, 5, bias, residual), act)
        _check(lib, *inputs(tokens, 264, 1000, F16, 6, bias, residual), act)


@pytest.mark.parametrize("tokens,cols,rows", [(4096, 136, 2320), (4100, 192, 2304), (2000, 4160, 40), (70, 200, 9000),
                                              (2048, 2560, 1024), (300, 9728, 640), (70, 40, 16401)])
def test_more_tiles_than_units_resident_and_splits(lib, tokens, cols, rows):
    _check(lib, *inputs(tokens, cols, rows, BF16, tokens), None)
    _check(lib, *inputs(tokens, cols, rows, F16, tokens), "gelu")


@pytest.mark.parametrize("cols", [64 * k for k in range(2, 17)])
def test_every_number_of_steps(lib, cols):
    _check(lib, *inputs(70, cols, 72, BF16, cols), "silu")
    _check(lib, *inputs(72, 72, cols, BF16, cols), None)


@pytest.mark.parametrize("tokens", [1, 5, 40, 150])
def test_strides_and_alignment(lib, tokens):
    for dtype, act in ((BF16, None), (F16, "silu")):
        x, W, b, r, dy = inputs(2 * tokens, 300, 150, dtype, tokens)
        for lo, hi in ((0, 264), (8, 272), (1, 257), (3, 203)):
            for at, n in ((7, 100), (8, 96)):
                ops = x[::2, lo:hi], W[10:10 + n, lo:hi], b[1:1 + n], r[1::2, at:at + n], dy[1::2, at:at + n]
                got = _check(lib, *ops, act)
                for a, c in zip(got, _check(lib, *(t.contiguous() for t in ops), act)):
                    assert torch.allclose(a.float(), c.float(), rtol=2 ** -6, atol=2e-2)


@pytest.mark.parametrize("tokens", [1, 16, 17, 32, 33, 70])
@pytest.mark.parametrize("cols,rows,lead", [(1, 1, 1), (7, 9, 3), (57, 130, 7), (65, 300, 0), (127, 300, 2), (1237, 260, 5)])
def test_rows_of_any_alignment_among_values_that_are_not_numbers(lib, tokens, cols, rows, lead):
    def inside(t, first, pad):
        buf = torch.full((first + t.shape[0] * (t.shape[1] + pad) + 8,), float("nan"), dtype=t.dtype, device="cuda")
        v = torch.as_strided(buf, t.shape, (t.shape[1] + pad, 1), first)
        v.copy_(t)
        return v
    for dtype, act in ((BF16, "silu"), (F16, None)):
        x, W, b, r, dy = inputs(tokens, cols, rows, dtype, tokens + cols)
        for pad in (0, 3):
            _check(lib, inside(x, 1, pad), inside(W, lead, pad), inside(b[None], 1, 0)[0], inside(r, lead, pad), inside(dy, 3, pad), act)


def test_empty_batch(lib):
    x, W, b, r, dy = inputs(4, 64, 32, BF16, 0)
    y, z = lib.linear_forward(x[:0], W, b, "silu", r[:0], save=True)
    assert y.shape == (0, 32) and z.shape == (0, 32)
    dx, dw, db = lib.linear_backward(x[:0], W, z, dy[:0], "silu")
    assert dx.shape == (0, 64) and dw.shape == W.shape and not dw.any() and not db.any()


def test_bad_token_stays_in_its_row(lib):
    for tokens in (6, 200):
        x, W, b, r, dy = inputs(tokens, 136, 72, BF16, 2)
        y = lib.linear_forward(x, W, b, "gelu", r)
        bad, rest = x.clone(), r.clone()
        bad[3, 100] = float("nan")
        rest[5] = float("inf")
        yb = lib.linear_forward(bad, W, b, "gelu", rest)
        keep = [t for t in range(tokens) if t not in (3, 5)]
        assert torch.equal(y[keep], yb[keep]) and torch.isnan(yb[3]).all() and torch.isinf(yb[5]).all()


def test_leading_dimensions_and_expanded_residual(lib):
    x, W, b, r, dy = inputs(24, 160, 96, F16, 3)
    wide = r[:1].expand(24, 96)
    y = lib.linear_forward(x.view(2, 3, 4, 160), W, b, None, wide.reshape(2, 3, 4, 96))
    assert y.shape == (2, 3, 4, 96) and torch.equal(y.view(24, 96), lib.linear_forward(x, W, b, None, wide.contiguous()))
    leaf = r[:1].clone().requires_grad_()
    lib.linear(x, W, b, None, leaf.expand(24, 96)).backward(dy)
    want = dy.double().sum(0, keepdim=True)
    assert bool(((leaf.grad.double() - want).abs() <= 2 * U[F16] * dy.double().abs().sum(0)).all())


def test_autograd(lib):
    for act in (None, "gelu"):
        x, W, b, r, dy = inputs(30, 64, 48, BF16, 7)
        y, z = lib.linear_forward(x, W, b, act, r, save=True)
        want = (*lib.linear_backward(x, W, z, dy, act), dy)
        leaves = [t.clone().requires_grad_() for t in (x, W, b, r)]
        out = lib.linear(leaves[0], leaves[1], leaves[2], act, leaves[3])
        assert torch.equal(out, y)
        out.backward(dy)
        assert all(torch.equal(t.grad, w) for t, w in zip(leaves, want))
        for k in range(4):   # one leaf at a time
            leaves = [t.clone().requires_grad_(i == k) for i, t in enumerate((x, W, b, r))]
            lib.linear(leaves[0], leaves[1], leaves[2], act, leaves[3]).backward(dy)
            assert [t.grad is not None for t in leaves] == [i == k for i in range(4)] and torch.equal(leaves[k].grad, want[k])
        leaves = [x.clone().requires_grad_(), W]
        lib.linear(*leaves, act=act).sum().backward()   # an expanded dy, no bias, no residual
        z = lib.linear_forward(x, W, None, act, save=True)[1]
        assert torch.equal(leaves[0].grad, lib.linear_backward(x, W, z, torch.ones_like(dy), act)[0])
        with torch.no_grad():
            assert not lib.linear(*leaves, act=act).requires_grad


def test_gradient_against_differences(lib):
    # sum(y dy) moves by <grad, step>; the kept fp32 z gives y here, since 16-bit outputs are too coarse
    x, W, b, r, dy = inputs(8, 64, 32, F16, 9)
    z = lib.linear_forward(x, W, b, "silu", save=True)[1]
    grads = lib.linear_backward(x, W, z, dy, "silu")

    def loss(*ops):
        z = lib.linear_forward(*ops, "silu", save=True)[1].double()
        return float((z * torch.sigmoid(z) * dy.double()).sum())
    for k, grad in enumerate(grads):
        ops = [x, W, b]
        step = torch.sign(torch.randn_like(grad.float())) * ops[k].float().abs().clamp(min=2 ** -6) * 2 ** -5
        hi, lo = [list(ops) for _ in range(2)]
        hi[k] = (ops[k].float() + step).to(F16)
        lo[k] = (ops[k].float() - step).to(F16)
        moves = grad.double() * (hi[k].double() - lo[k].double())
        # third-order term of a 1/32 relative step, against the terms' root sum of squares
        assert abs(loss(*hi) - loss(*lo) - float(moves.sum())) <= 0.05 * float(moves.norm()) + 1e-3 * abs(float(moves.sum())), k


@pytest.mark.parametrize("tokens", [3, 50, 500])
def test_fp16_gradients_in_range_neither_overflow_nor_vanish(lib, tokens):
    # rows of dy that differ by 2^20: dz is held with a scale for each row of an output
    x, W, b, r, dy = inputs(tokens, 96, 128, F16, 3)
    size = torch.logspace(-4, 4, tokens, device="cuda")[:, None]
    dy = (dy.float() * size).half()
    y, z = lib.linear_forward(x, W, b, "silu", save=True)
    dx = lib.linear_backward(x, W, z, dy, "silu")[0]
    ref = gradient_checks(x, W, b, dy, "silu")[0][1]
    keep = (ref.abs() > 2.0 ** -14) & (ref.abs() < 60000)
    row = ref.abs().amax(1, keepdim=True)
    assert bool(((dx.double() - ref).abs()[keep] <= (U[F16] * ref.abs() + 2e-5 * row)[keep]).all())


@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("tokens,cols,rows", [(70, 136, 72), (70, 135, 71), (32, 9728, 300), (200, 4096, 72)])
def test_workspace(lib, act, tokens, cols, rows):
    x, W, b, r, dy = inputs(tokens, cols, rows, BF16, 8)
    aligned = cols % 8 == 0 and rows % 8 == 0
    y, z = lib.linear_forward(x, W, b, act, r, save=True)
    want = lib.linear_backward(x, W, z, dy, act)
    need = lib.linear_backward_workspace_bytes(tokens, cols, rows, act, aligned)
    assert need <= lib.linear_backward_workspace_bytes(tokens, cols, rows, act, False)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    got = lib.linear_backward(x, W, z, dy, act, workspace=ws[:need])
    assert all(torch.equal(a, c) for a, c in zip(got, want)) and bool((ws[need:] == 0xFF).all())
    if need > 512:
        with pytest.raises(lib.ExterndError):
            lib.linear_backward(x, W, z, dy, act, workspace=ws[:256])
    n = lib.linear_forward_workspace_bytes(tokens, cols, rows, cols % 8 == 0)
    assert n <= lib.linear_forward_workspace_bytes(tokens, cols, rows, False)
    ws = torch.full((n + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(lib.linear_forward(x, W, b, act, r, workspace=ws[:n]), y) and bool((ws[n:] == 0xFF).all())
    out = torch.empty_like(y)
    assert lib.linear_forward(x, W, b, act, r, out=out) is out and torch.equal(out, y)


def test_side_stream(lib):
    x, W, b, r, dy = inputs(128, 256, 192, BF16, 8)
    y, z = lib.linear_forward(x, W, b, "silu", r, save=True)
    want = lib.linear_backward(x, W, z, dy, "silu")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        late = torch.zeros_like(x)
        late.copy_(x)
        y2, z2 = lib.linear_forward(late, W, b, "silu", r, save=True)
        got = lib.linear_backward(late, W, z2, dy, "silu")
    s.synchronize()
    assert torch.equal(y2, y) and all(torch.equal(a, c) for a, c in zip(got, want))


@pytest.mark.parametrize("tokens", [2, 150])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_in_a_graph(lib, tokens, dtype):
    x, W, b, r, dy = inputs(tokens, 256, 192, dtype, 8)
    lib.linear_backward(x, W, lib.linear_forward(x, W, b, "silu", r, save=True)[1], dy, "silu")
    torch.cuda.synchronize()
    static, grad = x.clone(), dy.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, z = lib.linear_forward(static, W, b, "silu", r, save=True)
        grads = lib.linear_backward(static, W, z, grad, "silu")
    for k in range(4):
        new = inputs(tokens, 256, 192, dtype, 20 + k)
        static.copy_(new[0])
        grad.copy_(new[4] * 2.0 ** (3 * k - 6))   # (other scales of dz in each replay)
        graph.replay()
        torch.cuda.synchronize()
        y2, z2 = lib.linear_forward(new[0], W, b, "silu", r, save=True)
        want = lib.linear_backward(new[0], W, z2, grad, "silu")
        assert torch.equal(y, y2) and all(torch.equal(a, c) for a, c in zip(grads, want))


def test_refusals(lib):
    x, W, b, r, dy = inputs(4, 64, 32, BF16, 0)
    for bad in (lambda: lib.linear_forward(x.float(), W.float()), lambda: lib.linear_forward(x, W.half()),
                lambda: lib.linear_forward(x, W.cpu()), lambda: lib.linear_forward(x, W, b.float())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: lib.linear_forward(x[:, :60], W), lambda: lib.linear_forward(x, W[0]), lambda: lib.linear_forward(x, W, b[:31]),
                lambda: lib.linear_forward(x, W, b, "relu"), lambda: lib.linear_forward(x, W, b, None, r[:3]),
                lambda: lib.linear_forward(x, W, b, None, r[:1]), lambda: lib.linear_forward(x, W, b, None, r.half()),
                lambda: lib.linear_forward(x, W, out=r[:3]), lambda: lib.linear_backward(x, W, None, dy[:3])):
        with pytest.raises(ValueError):
            bad()
    z = lib.linear_forward(x, W, b, "silu", save=True)[1]
    with pytest.raises(ValueError):
        lib.linear_backward(x, W, z[:3].contiguous(), dy, "silu")
    with pytest.raises(TypeError):
        lib.linear_backward(x, W, z.half(), dy, "silu")
    with pytest.raises(TypeError):
        lib.linear_backward(x, W, None, dy, "silu")
    with pytest.raises(TypeError):
        lib.linear_backward(x, W, z, dy.float(), "silu")
    with pytest.raises(lib.ExterndError, match="overlaps"):
        lib.linear_forward(x, W, b, None, r, out=r)
    square = torch.randn(64, 64, device="cuda").bfloat16()
    keep = x.clone()
    with pytest.raises(lib.ExterndError, match="overlaps"):
        lib.linear_forward(x, square, out=x)
    assert torch.equal(x, keep)
    leaf = W.clone().requires_grad_()
    with pytest.raises(RuntimeError, match="linear has"):
        lib.linear_forward(x, leaf).float().sum().backward()
    with pytest.raises(RuntimeError, match="out"):
        lib.linear_forward(x, leaf, out=torch.empty_like(r))
