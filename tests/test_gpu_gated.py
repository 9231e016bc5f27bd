"""GPU checks of the gated feed-forward block, forward and backward, against
oracle/gated.py in fp64.

Tolerances.  Operands are 16-bit, products exact in fp32, sums fp32: a sum of n
terms of total magnitude S is off by at most (n + 64) 2^-24 S.  h, dx, dWg and dWu are
rounded once to the operands' type (half ulp u: 2^-8 bf16, 2^-11 fp16), dg and
du before the products by the same u, which moves a gradient by at most u times
its terms' total magnitude.  Activation values and slopes are Lipschitz with
constants below 1.13 and 0.9 and carry a few fp32 roundings of their own.
fp16 adds its subnormal step."""
import numpy as np
import pytest
import torch

from oracle import gated as og

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}
E = 2.0 ** -24


def _host(t):
    return t.detach().cpu().double().numpy()


def _inputs(tokens, cols, rows, dtype, seed):
    rng = np.random.default_rng(seed)
    t = lambda a: torch.from_numpy(a.astype(np.float32)).to(dtype).cuda()
    scale = 1.0 / np.sqrt(cols)
    return (t(rng.standard_normal((tokens, cols))), t(scale * 1.5 * rng.standard_normal((rows, cols))),
            t(scale * rng.standard_normal((rows, cols))), t(rng.standard_normal((tokens, rows))))


def _projection_errors(x, wg, wu):
    cols = x.shape[1]
    return (cols + 64) * E * (np.abs(x) @ np.abs(wg).T), (cols + 64) * E * (np.abs(x) @ np.abs(wu).T)


def _within(got, ref, tol, what):
    err = np.abs(_host(got).reshape(ref.shape) - ref)
    assert np.all(err <= tol), (what, float((err / tol).max()))


def _check(lib, tokens, cols, rows, dtype, act, seed, tensors=None):
    xt, wgt, wut, dht = tensors or _inputs(tokens, cols, rows, dtype, seed)
    x, wg, wu, dh = map(_host, (xt, wgt, wut, dht))
    h, g, u = lib.gated_forward(xt, wgt, wut, act, save=True)
    assert torch.equal(lib.gated_forward(xt, wgt, wut, act), h)
    ref, gv, uv = og.forward(x, wg, wu, act)
    eg, eu = _projection_errors(x, wg, wu)
    _within(g, gv, eg + 1e-30, "g")
    _within(u, uv, eu + 1e-30, "u")
    a, slope = og.act(act, gv)
    ea, es = 1.13 * eg + 16 * E * np.abs(gv), 0.9 * eg + 32 * E * (1 + np.abs(gv))
    un, tiny = U[dtype] * 1.02, TINY[dtype]
    _within(h, ref, ea * (np.abs(uv) + eu) + np.abs(a) * eu + un * np.abs(ref) + tiny, "h")

    dx, dwg, dwu = lib.gated_backward(xt, wgt, wut, g, u, dht, act)
    dg, du = dh * uv * slope, dh * a
    edg = np.abs(dh) * ((np.abs(uv) + eu) * es + eu * np.abs(slope)) + un * np.abs(dg) + tiny
    edu = np.abs(dh) * ea + un * np.abs(du) + tiny
    rdx, rdg, rdu = og.backward(x, wg, wu, dh, act)
    mdx = (np.abs(dg) + edg) @ np.abs(wg) + (np.abs(du) + edu) @ np.abs(wu)
    _within(dx, rdx, edg @ np.abs(wg) + edu @ np.abs(wu) + (2 * rows + 128) * E * mdx + un * np.abs(rdx) + tiny, "dx")
    for got, want, d, ed, what in ((dwg, rdg, dg, edg, "dWg"), (dwu, rdu, du, edu, "dWu")):
        m = (np.abs(d) + ed).T @ np.abs(x)
        _within(got, want, ed.T @ np.abs(x) + (tokens + 64) * E * m + un * np.abs(want) + tiny, what)
    return h, dx, dwg, dwu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,cols,rows", [
    (1, 1, 1), (1, 64, 128), (3, 8, 16), (2, 7, 5), (16, 128, 64), (17, 72, 40), (33, 200, 136), (64, 256, 512),
    (65, 333, 129), (100, 1000, 24), (130, 63, 65), (257, 264, 300), (300, 520, 1032), (600, 77, 131)])
def test_block(lib, dtype, tokens, cols, rows):
    act = ("silu", "gelu", "gelu_tanh")[(tokens + cols) % 3]
    _check(lib, tokens, cols, rows, dtype, act, tokens + rows)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations(lib, act):
    _check(lib, 40, 96, 80, torch.bfloat16, act, 5)
    _check(lib, 200, 96, 80, torch.float16, act, 6)


def test_wide_projections_stay_finite(lib):
    x, wg, wu, dh = _inputs(70, 64, 48, torch.bfloat16, 1)
    x = x * 3000
    for act in ("silu", "gelu", "gelu_tanh"):
        h, g, u = lib.gated_forward(x, wg, wu, act, save=True)
        grads = lib.gated_backward(x, wg, wu, g, u, dh, act)
        assert all(torch.isfinite(t).all() for t in (h, *grads))
        assert (g < -200).any() and (h[g < -200] == 0).all()


@pytest.mark.parametrize("tokens", [1, 5, 40, 150])
def test_strides_and_alignment(lib, tokens):
    dtype = torch.bfloat16
    x, wg, wu, dh = _inputs(2 * tokens, 300, 150, dtype, tokens)
    for lo, hi in ((0, 264), (8, 272), (1, 257), (3, 203)):
        xs, gs, us, ds = x[::2, lo:hi], wg[10:110, lo:hi], wu[40:140, lo:hi], dh[1::2, 7:107]
        got = _check(lib, tokens, hi - lo, 100, dtype, "silu", 0, (xs, gs, us, ds))
        same = [t.contiguous() for t in (xs, gs, us, ds)]
        want = _check(lib, tokens, hi - lo, 100, dtype, "silu", 0, same)
        for a, b in zip(got, want):
            assert torch.allclose(a.float(), b.float(), rtol=2 ** -6, atol=1e-2)


def test_shared_packed_weights(lib):
    # gate and up halves of one matrix, and leading batch dimensions
    x, wg, wu, dh = _inputs(24, 160, 96, torch.float16, 3)
    both = torch.cat([wg, wu])
    h = lib.gated_forward(x.view(2, 3, 4, 160), both[:96], both[96:])
    assert h.shape == (2, 3, 4, 96)
    assert torch.equal(h.view(24, 96), lib.gated_forward(x, wg, wu))


def test_empty_batch(lib):
    x, wg, wu, dh = _inputs(4, 64, 32, torch.bfloat16, 0)
    h, g, u = lib.gated_forward(x[:0], wg, wu, save=True)
    assert h.shape == (0, 32) and g.shape == (0, 32)
    dx, dwg, dwu = lib.gated_backward(x[:0], wg, wu, g, u, dh[:0])
    assert dx.shape == (0, 64) and not dwg.any() and not dwu.any()


def test_bad_token_stays_in_its_row(lib):
    for tokens in (6, 200):
        x, wg, wu, dh = _inputs(tokens, 136, 72, torch.bfloat16, 2)
        h = lib.gated_forward(x, wg, wu)
        bad = x.clone()
        bad[3, 100] = float("nan")
        bad[5, 0] = float("inf")
        hb = lib.gated_forward(bad, wg, wu)
        keep = [t for t in range(tokens) if t not in (3, 5)]
        assert torch.equal(h[keep], hb[keep])
        assert torch.isnan(hb[3]).all() and not torch.isfinite(hb[5]).any()


def test_parts_of_the_gradient(lib):
    x, wg, wu, dh = _inputs(50, 128, 64, torch.bfloat16, 4)
    h, g, u = lib.gated_forward(x, wg, wu, save=True)
    dx, dwg, dwu = lib.gated_backward(x, wg, wu, g, u, dh)
    a = lib.gated_backward(x, wg, wu, g, u, dh, need_dw=False)
    b = lib.gated_backward(x, wg, wu, g, u, dh, need_dx=False)
    assert torch.equal(a[0], dx) and a[1] is None and a[2] is None
    assert b[0] is None and torch.equal(b[1], dwg) and torch.equal(b[2], dwu)
    again = lib.gated_backward(x, wg, wu, g, u, dh)
    assert all(torch.equal(p, q) for p, q in zip(again, (dx, dwg, dwu)))


def test_autograd(lib):
    x, wg, wu, dh = _inputs(30, 64, 48, torch.bfloat16, 7)
    h, g, u = lib.gated_forward(x, wg, wu, "gelu", save=True)
    want = lib.gated_backward(x, wg, wu, g, u, dh, "gelu")
    leaves = [t.clone().requires_grad_() for t in (x, wg, wu)]
    out = lib.gated(*leaves, "gelu")
    assert torch.equal(out, h)
    out.backward(dh)
    assert all(torch.equal(t.grad, w) for t, w in zip(leaves, want))
    leaves = [x.clone().requires_grad_(), wg, wu]
    lib.gated(*leaves).sum().backward()   # an expanded dh
    ones = torch.ones_like(dh)
    h, g, u = lib.gated_forward(x, wg, wu, save=True)
    assert torch.equal(leaves[0].grad, lib.gated_backward(x, wg, wu, g, u, ones)[0])


def test_gradient_against_differences(lib):
    # sum(h dh) moves by <grad, step>: the kernel's own forward in fp16 outputs is
    # too coarse, so the kept fp32 projections give h here
    x, wg, wu, dh = _inputs(8, 64, 32, torch.float16, 9)
    h, g, u = lib.gated_forward(x, wg, wu, save=True)
    dx, dwg, dwu = lib.gated_backward(x, wg, wu, g, u, dh)

    def loss(*ops):
        _, gg, uu = lib.gated_forward(*ops, save=True)
        return float((gg.double() * torch.sigmoid(gg.double()) * uu.double() * dh.double()).sum())
    for k, grad in enumerate((dx, dwg, dwu)):
        ops = [x, wg, wu]
        step = torch.sign(torch.randn_like(grad.float())) * ops[k].float().abs().clamp(min=2 ** -6) * 2 ** -5
        hi, lo = [list(ops) for _ in range(2)]
        hi[k] = (ops[k].float() + step).to(ops[k].dtype)
        lo[k] = (ops[k].float() - step).to(ops[k].dtype)
        diff = loss(*hi) - loss(*lo)
        want = float((grad.double() * (hi[k].double() - lo[k].double())).sum())
        # third-order term of a 1/32 relative step, against the terms' root sum of squares
        size = float((grad.double() * (hi[k].double() - lo[k].double())).norm())
        assert abs(diff - want) <= 0.05 * size + 1e-3 * abs(want), k


def test_workspace(lib):
    x, wg, wu, dh = _inputs(70, 136, 72, torch.bfloat16, 8)
    h, g, u = lib.gated_forward(x, wg, wu, save=True)
    want = lib.gated_backward(x, wg, wu, g, u, dh)
    need = lib.gated_backward_workspace_bytes(70, 136, 72)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    got = lib.gated_backward(x, wg, wu, g, u, dh, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(lib.ExterndError):
        lib.gated_backward(x, wg, wu, g, u, dh, workspace=ws[:need // 2])
    n = lib.gated_forward_workspace_bytes(70, 136, 72)
    ws = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(lib.gated_forward(x, wg, wu, workspace=ws), h)


def test_side_stream(lib):
    x, wg, wu, dh = _inputs(128, 256, 192, torch.bfloat16, 8)
    h, g, u = lib.gated_forward(x, wg, wu, save=True)
    want = lib.gated_backward(x, wg, wu, g, u, dh)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        late = torch.zeros_like(x)
        late.copy_(x)
        h2, g2, u2 = lib.gated_forward(late, wg, wu, save=True)
        got = lib.gated_backward(late, wg, wu, g2, u2, dh)
    s.synchronize()
    assert torch.equal(h2, h) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("tokens", [2, 150])
def test_in_a_graph(lib, tokens):
    x, wg, wu, dh = _inputs(tokens, 256, 192, torch.bfloat16, 8)
    lib.gated_backward(x, wg, wu, *lib.gated_forward(x, wg, wu, save=True)[1:], dh)
    torch.cuda.synchronize()
    ws = torch.empty((lib.gated_backward_workspace_bytes(tokens, 256, 192),), dtype=torch.uint8, device="cuda")
    static = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, g, u = lib.gated_forward(static, wg, wu, save=True)
        grads = lib.gated_backward(static, wg, wu, g, u, dh, workspace=ws)
    for k in range(4):
        new = _inputs(tokens, 256, 192, torch.bfloat16, 20 + k)[0]
        static.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        h2, g2, u2 = lib.gated_forward(new, wg, wu, save=True)
        want = lib.gated_backward(new, wg, wu, g2, u2, dh)
        assert torch.equal(h, h2) and all(torch.equal(a, b) for a, b in zip(grads, want))


def test_refusals(lib):
    x, wg, wu, dh = _inputs(4, 64, 32, torch.bfloat16, 0)
    with pytest.raises(TypeError):
        lib.gated_forward(x.float(), wg.float(), wu.float())
    with pytest.raises(TypeError):
        lib.gated_forward(x, wg, wu.half())
    with pytest.raises(TypeError):
        lib.gated_forward(x, wg, wu.cpu())
    with pytest.raises(ValueError):
        lib.gated_forward(x, wg, wu[:31])
    with pytest.raises(ValueError):
        lib.gated_forward(x[:, :60], wg, wu)
    with pytest.raises(ValueError):
        lib.gated_forward(x, wg, wu, "relu")
    h, g, u = lib.gated_forward(x, wg, wu, save=True)
    with pytest.raises(ValueError):
        lib.gated_backward(x, wg, wu, g, u, dh[:3])
    with pytest.raises(ValueError):
        lib.gated_backward(x, wg, wu, g[:3].contiguous(), u, dh)
    with pytest.raises(TypeError):
        lib.gated_backward(x, wg, wu, g.half(), u, dh)
    with pytest.raises(TypeError):
        lib.gated_backward(x, wg, wu, g, u, dh.float())


@pytest.mark.parametrize("cols", [64 * k for k in range(2, 17)])
def test_every_number_of_steps(lib, cols):
    # the contraction's loop begins, repeats after six steps and ends at every phase
    _check(lib, 70, cols, 72, torch.bfloat16, "silu", cols)


@pytest.mark.parametrize("tokens,cols,rows", [(4096, 136, 2320), (4100, 192, 2304), (2000, 4160, 40), (70, 200, 9000)])
def test_more_tiles_than_units_resident(lib, tokens, cols, rows):
    # workgroups that take several tiles, contractions split over workgroups, both tile sizes
    _check_on_device(lib, tokens, cols, rows, torch.bfloat16, "silu")
    _check_on_device(lib, tokens, cols, rows, torch.float16, "gelu")


def _check_on_device(lib, tokens, cols, rows, dtype, act):
    """As _check, with the fp64 reference on the device (the shapes are too large for the host)."""
    x, wg, wu, dh = _inputs(tokens, cols, rows, dtype, tokens)
    X, G, U_, D = (t.double() for t in (x, wg, wu, dh))
    gv, uv = X @ G.t(), X @ U_.t()
    a, slope = (torch.from_numpy(t).cuda() for t in og.act(act, _host(gv)))
    eg, eu = (cols + 64) * E * (X.abs() @ G.abs().t()), (cols + 64) * E * (X.abs() @ U_.abs().t())
    ea, es = 1.13 * eg + 16 * E * gv.abs(), 0.9 * eg + 32 * E * (1 + gv.abs())
    un, tiny = U[dtype] * 1.02, TINY[dtype]
    h, g, u = lib.gated_forward(x, wg, wu, act, save=True)
    dx, dwg, dwu = lib.gated_backward(x, wg, wu, g, u, dh, act)
    ref = a * uv
    dg, du = D * uv * slope, D * a
    edg = D.abs() * ((uv.abs() + eu) * es + eu * slope.abs()) + un * dg.abs() + tiny
    edu = D.abs() * ea + un * du.abs() + tiny
    rows_of = lambda d, e: d.abs() + e
    checks = [("g", g, gv, eg + 1e-30), ("u", u, uv, eu + 1e-30),
              ("h", h, ref, ea * (uv.abs() + eu) + a.abs() * eu + un * ref.abs() + tiny)]
    want = dg @ G + du @ U_
    mdx = rows_of(dg, edg) @ G.abs() + rows_of(du, edu) @ U_.abs()
    checks.append(("dx", dx, want,
                   edg @ G.abs() + edu @ U_.abs() + (2 * rows + 128) * E * mdx + un * want.abs() + tiny))
    for name, got, d, e in (("dWg", dwg, dg, edg), ("dWu", dwu, du, edu)):
        want = d.t() @ X
        m = rows_of(d, e).t() @ X.abs()
        checks.append((name, got, want, e.t() @ X.abs() + (tokens + 64) * E * m + un * want.abs() + tiny))
    for name, got, want, tol in checks:
        err = (got.double() - want).abs()
        assert bool((err <= tol).all()), (name, float((err / tol).max()))


@pytest.mark.parametrize("tokens", [16, 17, 32, 33])
@pytest.mark.parametrize("cols,rows", [(5000, 40), (5008, 40), (5001, 24), (9736, 72), (1024, 21008)])
def test_token_counts_where_the_form_changes(lib, tokens, cols, rows):
    # few tokens take one kernel, more of them another, by the columns a compute unit reads
    _check_on_device(lib, tokens, cols, rows, torch.bfloat16, "silu")
    _check_on_device(lib, tokens, cols, rows, torch.float16, "gelu_tanh")


@pytest.mark.parametrize("tokens", [1, 16, 17, 32])
@pytest.mark.parametrize("cols,rows,lead", [(1, 1, (1, 1)), (7, 9, (3, 3)), (57, 130, (7, 0)), (64, 17, (5, 5)),
                                            (65, 300, (0, 1)), (121, 129, (1, 7)), (127, 300, (2, 2)),
                                            (1237, 260, (0, 0)), (2559, 4200, (0, 0)), (2001, 4200, (6, 3))])
def test_few_tokens_on_rows_of_any_alignment(lib, tokens, cols, rows, lead):
    # what lies around the operands is NaN, and each starts at its own distance from 16 bytes
    def inside(t, first, pad):
        buf = torch.full((first + t.shape[0] * (t.shape[1] + pad) + 8,), float("nan"), dtype=t.dtype, device="cuda")
        v = torch.as_strided(buf, t.shape, (t.shape[1] + pad, 1), first)
        v.copy_(t)
        return v
    for dtype, act in ((torch.bfloat16, "silu"), (torch.float16, "gelu")):
        x, wg, wu, dh = _inputs(tokens, cols, rows, dtype, tokens + cols)
        want = lib.gated_forward(torch.nn.functional.pad(x, (0, -cols % 8)), torch.nn.functional.pad(wg, (0, -cols % 8)),
                                 torch.nn.functional.pad(wu, (0, -cols % 8)), act, save=True)
        for pad in (0, 3):
            got = lib.gated_forward(inside(x, 1, pad), inside(wg, lead[0], pad), inside(wu, lead[1], pad), act, save=True)
            X, G, U_ = (t.double() for t in (x, wg, wu))
            for g, W in ((got[1], G), (got[2], U_)):
                tol = (cols + 64) * E * (X.abs() @ W.abs().t()) + 1e-30
                assert bool(((g.double() - X @ W.t()).abs() <= tol).all())
            # the projections differ by the order of their sums only, and h by what that does to it
            tol = 3 * (cols + 64) * E * ((X.abs() @ G.abs().t()) * (U_.abs() @ X.abs().t()).t() * 2.26 +
                                         (X.abs() @ G.abs().t())) + 64 * E * want[0].double().abs()
            un = 2 * 1.02 * U[dtype] * want[0].double().abs() + 2 * TINY[dtype]
            assert bool(((got[0].double() - want[0].double()).abs() <= tol + un).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,cols,rows", [(1, 64, 40), (2, 470, 2211), (33, 130, 63), (64, 200, 640), (5, 33000, 72)])
def test_few_tokens_dx_is_rounded_once(lib, dtype, tokens, cols, rows):
    # dg and du enter dx with both of their 16-bit parts: what is left of their rounding is its square
    x, wg, wu, dh = _inputs(tokens, cols, rows, dtype, cols)
    X, G, U_, D = (t.double() for t in (x, wg, wu, dh))
    gv, uv = X @ G.t(), X @ U_.t()
    a, slope = (torch.from_numpy(t).cuda() for t in og.act("gelu", _host(gv)))
    eg, eu = (cols + 64) * E * (X.abs() @ G.abs().t()), (cols + 64) * E * (X.abs() @ U_.abs().t())
    ea, es = 1.13 * eg + 16 * E * gv.abs(), 0.9 * eg + 32 * E * (1 + gv.abs())
    un, tiny = U[dtype] * 1.02, TINY[dtype]
    parts = un ** 2 if cols <= 32768 else un   # (wider than that, one part is kept)
    dg, du = D * uv * slope, D * a
    edg = D.abs() * ((uv.abs() + eu) * es + eu * slope.abs()) + parts * dg.abs() + tiny
    edu = D.abs() * ea + parts * du.abs() + tiny
    _, g, u = lib.gated_forward(x, wg, wu, "gelu", save=True)
    dx, _, _ = lib.gated_backward(x, wg, wu, g, u, dh, "gelu")
    want = dg @ G + du @ U_
    m = (dg.abs() + edg) @ G.abs() + (du.abs() + edu) @ U_.abs()
    tol = edg @ G.abs() + edu @ U_.abs() + (4 * rows + 128) * E * m + un * want.abs() + tiny
    assert bool(((dx.double() - want).abs() <= tol).all())


def test_few_tokens_overflow_stays_infinite(lib):
    # a dg past fp16's range is infinite in its first part, and the second adds nothing to that
    x, wg, wu, dh = _inputs(2, 64, 40, torch.float16, 3)
    wg, wu, x = wg.abs() + 1, wu.abs() + 1, x.abs() + 1
    dh = torch.full_like(dh, 60000.0)
    _, g, u = lib.gated_forward(x, wg, wu, "silu", save=True)
    dx, _, _ = lib.gated_backward(x, wg, wu, g, u, dh, "silu")
    assert bool(torch.isinf(dx).all()) and bool((dx > 0).all())
