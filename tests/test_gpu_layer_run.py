"""The gated block, the linear layer, the optimizer and the experts run together, as training steps and as a decoding loop
do, eagerly and from a graph.

Every operator of a run is checked at the operands it had in that run, by the bounds derived in
tests/linear_reference.py, tests/test_gpu_moe.py and tests/gated_reference.py; what autograd or a graph gives has to be
the operators' own results bit by bit."""
import importlib.util
import os

import pytest
import torch

import gated_reference
import linear_reference
from test_gpu_moe import _bound, _check_experts
from test_gpu_moe import _inputs as moe_inputs

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F16 = torch.bfloat16, torch.float16


def _mlp(dtype, tokens, cols, rows, seed):
    """x, target, [Wg, Wu, Wd, bias]."""
    x, wg, wu, _ = gated_reference.inputs(tokens, cols, rows, dtype, seed)
    _, wd, bias, target, _ = linear_reference.inputs(tokens, rows, cols, dtype, seed + 1)
    return x, target, [wg, wu, wd, bias]


def _loss(lib, x, target, params):
    wg, wu, wd, bias = params
    h = lib.gated(x, wg, wu)
    y = lib.linear(h, wd, bias, None, x)
    return h, y, 2.0 * (y.float() - target.float()).square().mean()


def _within(got, want, tol, name):
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), (name, float((err / tol).max()))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("tokens,cols,rows", [(1, 64, 48), (5, 72, 130), (40, 131, 77), (300, 264, 520)])
def test_gradients_of_a_block(lib, dtype, tokens, cols, rows):
    x, target, params = _mlp(dtype, tokens, cols, rows, tokens)
    wg, wu, wd, bias = params
    leaves = [p.clone().requires_grad_() for p in (x, *params)]
    h, y, loss = _loss(lib, leaves[0], target, leaves[1:])
    h.retain_grad()
    y.retain_grad()
    scale = 2.0 ** 10   # dy of a mean is small: fp16's gradients of it need a scale
    (loss * scale).backward()
    dy, dh = y.grad, h.grad
    h, y = h.detach(), y.detach()
    # the linear layer at h, x as its residual
    for got, (name, want, tol) in zip((y,), linear_reference.forward_checks(h, wd, bias, None, x)[1:]):
        _within(got, want, tol, name)
    for got, (name, want, tol) in zip((dh, leaves[3].grad, leaves[4].grad), linear_reference.gradient_checks(h, wd, bias, dy, None)):
        _within(got, want, tol, name)
    # the gated block at dh; x's gradient is the block's, rounded, and the residual's dy, rounded again together
    u = 1.02 * gated_reference.U[dtype]
    tiny = gated_reference.TINY[dtype]
    step = None if dtype == BF16 else tiny
    for got, (name, want, tol) in zip((leaves[0].grad, leaves[1].grad, leaves[2].grad), gated_reference.references(x, wg, wu, dh, "silu", step)):
        tol = tol + u * (want.abs() + tol) + tiny
        if name == "dx":
            want = want + dy.double()
            tol = tol + u * (want.abs() + tol) + tiny
        _within(got, want, tol, name)


@pytest.mark.parametrize("dtype,bits,master", [(BF16, 32, False), (BF16, 8, True), (F16, 8, True), (F16, 32, True)])
def test_training_steps_eager_and_from_a_graph(lib, dtype, bits, master):
    x, target, params = _mlp(dtype, 96, 72, 200, 3)
    scale = 2.0 ** 10

    def make():
        # a run's parameters, optimizer and step; the gradients are asked for, not accumulated in the leaves
        mine = [p.clone().requires_grad_() for p in params]
        opt = lib.AdamW(mine, lr=1e-2, weight_decay=[0.1, 0.1, 0.1, 0.0], bits=bits, master=master)

        def step(x, target):
            loss = _loss(lib, x, target, mine)[2]
            opt.step(torch.autograd.grad(loss * scale, mine), grad_scale=1 / scale)
            return loss.detach()
        return mine, opt, step
    mine, opt, step = make()
    inputs = [_mlp(dtype, 96, 72, 200, 50 + k)[:2] for k in range(5)]
    losses, after = [], []
    for a, b in inputs:
        losses.append(step(a, b).clone())
        after.append([p.detach().clone() for p in mine])
    assert all(bool((p != q).any()) for p, q in zip(after[0], after[1]))

    again, opt2, step2 = make()
    sx, st = x.clone(), target.clone()
    sx.copy_(inputs[0][0])
    st.copy_(inputs[0][1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):   # the first step outside the graph
        first = step2(sx, st).clone()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(first, losses[0]) and all(torch.equal(p, q) for p, q in zip(again, after[0]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = step2(sx, st)
    for k in range(1, 5):
        sx.copy_(inputs[k][0])
        st.copy_(inputs[k][1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, losses[k]) and all(torch.equal(p, q) for p, q in zip(again, after[k])), k
    for a, b in zip(opt.state.values(), opt2.state.values()):
        assert a is None and b is None or torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("tokens", [1, 3, 20])
def test_decoding_through_experts(lib, dtype, tokens):
    # projection with a residual, experts restored from 4-bit codes, and the output's projection, three tokens in turn
    cols, rows, experts, top = 136, 72, 6, 2
    x, Wr, Wg, Wu, Wd = moe_inputs(tokens, cols, rows, experts, dtype, 40 + tokens)
    four = lambda w: torch.stack([lib.q4_reconstruct(lib.q4_quantize(e.float(), 32, symmetric=False), dtype) for e in w])
    Wg, Wu, Wd = four(Wg), four(Wu), four(Wd)
    _, wi, bi, _, _ = linear_reference.inputs(tokens, cols, cols, dtype, 7)
    _, wo, _, _, _ = linear_reference.inputs(tokens, cols, 300, dtype, 8, bias=False)

    def layer(x):
        a = lib.linear_forward(x, wi, bi, "gelu", x)
        m, ids, weights = lib.moe(a, Wr, Wg, Wu, Wd, top, routing=True)
        return a, ids, weights, m, lib.linear_forward(m, wo)

    def check(x, a, ids, weights, m, y):
        _within(a, *linear_reference.forward_checks(x, wi, bi, "gelu", x)[1][1:], "a")
        _check_experts(lib, m, a, ids, weights, Wg, Wu, Wd, "silu")
        _within(y, *linear_reference.forward_checks(m, wo, None, None, None)[1][1:], "y")
    check(x, *layer(x))
    static = x.clone()
    graphs = []
    for _ in range(2):   # two graphs of the same weights, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = layer(static)
        graphs.append((graph, got))
    for k in range(4):
        static.copy_(moe_inputs(tokens, cols, rows, experts, dtype, 60 + k)[0])
        graph, got = graphs[k % 2]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, layer(static))), k
    check(static, *got)


def test_example_trains_its_output_projection(lib):
    # the example runs, and its gradients are the operators' own
    spec = importlib.util.spec_from_file_location("compressed_mlp", os.path.join(ROOT, "examples", "compressed_mlp.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    x, target, (wg, wu, wd, _) = _mlp(BF16, 64, 96, 128, 9)
    wg, wu = mod.tune(x, lib.gated_forward(x, wg, wu), wg, wu, 32, 2, 1e-3)
    assert wg.dtype == torch.float32 and bool(torch.isfinite(wg).all()) and bool(torch.isfinite(wu).all())
    h = lib.gated_forward(x, wg.bfloat16(), wu.bfloat16())
    leaf = wd.clone().requires_grad_()
    grad, = torch.autograd.grad(mod.output_loss(h, leaf, target), leaf)
    y = lib.linear_forward(h, wd).float()
    dy = (2 * (y - target.float()) / y.numel() / target.float().square().mean()).bfloat16()
    _within(grad, *linear_reference.gradient_checks(h, wd, None, dy, None)[1][1:], "dWd")
    new = mod.tune_output(h, target, wd, 3, 1e-3)
    assert new.dtype == BF16 and new.shape == wd.shape and bool((new != wd).any()) and bool(torch.isfinite(new).all())


def test_one_expert_is_the_gated_block_and_the_linear_layer(lib):
    host = lambda t: t.cpu().double().numpy()
    # one expert of weight 1: h is rounded between the block and the layer, and kept in two parts by the experts
    for dtype in (BF16, F16):
        x, Wr, Wg, Wu, Wd = moe_inputs(6, 136, 72, 1, dtype, 5)
        y, ids, weights = lib.moe(x, Wr, Wg, Wu, Wd, 1, routing=True)
        assert not ids.any() and bool((weights == 1).all())
        h = lib.gated_forward(x, Wg[0], Wu[0])
        z = lib.linear_forward(h, Wd[0])
        _check_experts(lib, y, x, ids, weights, Wg, Wu, Wd, "silu")
        want, tol = (torch.from_numpy(t).cuda() for t in _bound(host(x), ids.cpu().numpy(),
                     host(weights), host(Wg), host(Wu), host(Wd), "silu", linear_reference.U[dtype], dtype))
        u, tiny = 1.02 * linear_reference.U[dtype], linear_reference.TINY[dtype]
        wd = Wd[0].double().abs()
        rounding = h.double().abs() @ wd.t() * u + tiny * wd.sum(1)
        _within(z, want, (tol + rounding) * (1 + 2 * u), "z")
