"""GPU checks of the mixture-of-experts layer against oracle/moe.py in fp64.

Tolerances.  Operands are 16-bit, products exact in fp32, sums fp32: n terms of total magnitude S are off by at
most (n + 64) 2^-24 S.  g and u are off by that, act(g) by 1.13 times as much and 16 roundings, h = act(g) u by their
product's.  h enters the second product in two parts, whose second is off by u^2 (u half a step of the type) and, in
fp16, by its subnormal step under the scaling, 2^-39 of the slot's largest.  y is the weighted sum of `top` slots in
fp32, each weight off by a few roundings (fp64 rounded once), and rounded once to the type.  The choice itself has to be
the oracle's: logits of random operands differ by far more than fp64 sums are off."""
import numpy as np
import pytest
import torch

from oracle import moe as om
from oracle.gated import act as oact

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11}
TINY = {BF16: 2.0 ** -133, F16: 2.0 ** -25}
E = 2.0 ** -24


def _host(t):
    return t.detach().cpu().double().numpy()


def _inputs(tokens, cols, rows, experts, dtype, seed, router=None):
    """x, Wr, Wg, Wu, Wd."""
    rng = np.random.default_rng(seed)
    t = lambda kind, s, *shape: torch.from_numpy((s * rng.standard_normal(shape)).astype(np.float32)).to(kind).cuda()
    s = 1 / np.sqrt(cols)
    return (t(dtype, 1.0, tokens, cols), t(router or dtype, s, experts, cols), t(dtype, 1.5 * s, experts, rows, cols),
            t(dtype, s, experts, rows, cols), t(dtype, 1 / np.sqrt(rows), experts, cols, rows))


def _bound(x, ids, weights, Wg, Wu, Wd, act, u, dtype):
    """(y, tolerance) in fp64."""
    y, tol = np.zeros_like(x), np.zeros_like(x)
    cols, rows = x.shape[1], Wg.shape[1]
    for t in range(x.shape[0]):
        for e, w in zip(ids[t], weights[t]):
            if not 0 <= e < Wg.shape[0]:
                continue
            g, v = Wg[e] @ x[t], Wu[e] @ x[t]
            eg, ev = (cols + 64) * E * (np.abs(Wg[e]) @ np.abs(x[t])), (cols + 64) * E * (np.abs(Wu[e]) @ np.abs(x[t]))
            a = oact(act, g)[0]
            ea = 1.13 * eg + 16 * E * np.abs(g)
            h = a * v
            eh = ea * (np.abs(v) + ev) + np.abs(a) * ev + 2 * E * np.abs(h)
            eh = eh + (1.02 * u) ** 2 * np.abs(h) + (np.abs(h).max(initial=0) * 2.0 ** -38 if dtype == F16 else TINY[dtype])
            m = np.abs(Wd[e]) @ (np.abs(h) + eh)
            y[t] += w * (Wd[e] @ h)
            tol[t] += abs(w) * (np.abs(Wd[e]) @ eh + (2 * rows + 128) * E * m + 8 * E * m)
    tol += len(ids[0]) * E * (np.abs(y) + tol)
    return y, tol + 1.02 * u * (np.abs(y) + tol) + TINY[dtype]


def _check_experts(lib, y, x, ids, weights, Wg, Wu, Wd, act):
    dtype = x.dtype
    cols = x.shape[-1]
    flat = lambda t: t.reshape(-1, t.shape[-1])
    want, tol = _bound(_host(flat(x)), flat(ids).cpu().numpy(), _host(flat(weights)), _host(Wg), _host(Wu), _host(Wd), act, U[dtype], dtype)
    err = np.abs(_host(y).reshape(want.shape) - want)
    assert np.all(err <= tol), float((err / tol).max())


def _check(lib, ops, top, act="silu", normalize=True):
    x, Wr, Wg, Wu, Wd = ops
    y, ids, weights = lib.moe(x, Wr, Wg, Wu, Wd, top, act, normalize, routing=True)
    want, w = om.route(_host(x), _host(Wr), top, normalize)
    assert np.array_equal(ids.cpu().numpy(), want)
    # a weight is a quotient of fp64 sums, rounded to fp32
    assert np.all(np.abs(_host(weights) - w) <= 1.01 * E * w)
    _check_experts(lib, y, x, ids, weights, Wg, Wu, Wd, act)
    alone = lib.moe_route(x, Wr, top, normalize)
    assert torch.equal(alone[0], ids) and torch.equal(alone[1], weights)
    assert torch.equal(lib.moe_experts(x, ids, weights, Wg, Wu, Wd, act), y)   # (the same kernels on the same slots)
    assert torch.equal(lib.moe(x, Wr, Wg, Wu, Wd, top, act, normalize), y)
    return y, ids, weights


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("tokens,cols,rows,experts,top", [
    (1, 1, 1, 1, 1), (1, 8, 8, 2, 2), (1, 64, 128, 4, 1), (3, 7, 5, 3, 2), (2, 72, 40, 16, 4), (5, 200, 136, 8, 8),
    (16, 130, 63, 13, 3), (17, 264, 33, 2, 1), (40, 96, 24, 4, 2), (64, 128, 16, 65, 6), (33, 65, 129, 129, 5),
    (4, 520, 16, 300, 10), (2, 1032, 24, 1024, 8), (1, 2304, 640, 6, 2), (200, 40, 24, 3, 2)])
def test_layer(lib, dtype, tokens, cols, rows, experts, top):
    ops = _inputs(tokens, cols, rows, experts, dtype, tokens + cols)
    _check(lib, ops, top, ("silu", "gelu", "gelu_tanh")[(cols + rows) % 3], normalize=tokens % 2 == 0)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("tokens,cols,rows,experts,top", [
    (8, 72, 40, 256, 8), (8, 72, 40, 257, 8), (8, 200, 33, 9, 8), (9, 72, 40, 256, 7), (8, 72, 40, 255, 9), (7, 71, 39, 256, 9),
    (2, 136, 48, 64, 32), (2, 136, 48, 64, 33), (1, 64, 40, 64, 64), (1, 64, 40, 65, 64), (1, 1000, 72, 1024, 64),
    (8, 64, 24, 2, 2), (8, 64, 24, 1, 1), (4, 8, 8, 16, 16), (4, 8, 8, 17, 17)])
def test_where_the_choices_are_made(lib, dtype, tokens, cols, rows, experts, top):
    # up to 8 tokens, 64 slots and 256 experts the first product makes them, past that a kernel of its own
    ops = _inputs(tokens, cols, rows, experts, dtype, tokens + experts)
    for normalize in (False, True):
        _check(lib, ops, top, "silu", normalize)


def test_few_tokens_that_choose_alike(lib):
    # all slots of a group: fewer experts than there may be groups; and every token its own experts
    x, Wr, Wg, Wu, Wd = _inputs(8, 64, 40, 32, BF16, 12)
    x = x.abs()
    for chosen in ([5, 9, 31], [0, 1, 2]):
        Wr[:] = -1
        for k, e in enumerate(chosen):
            Wr[e] = 2.0 ** -k
        ids = _check(lib, (x, Wr, Wg, Wu, Wd), 3)[1]
        assert bool((ids == torch.tensor(chosen, device="cuda", dtype=torch.int32)).all())
    Wr[:] = 0
    x[:] = 0
    for t in range(8):
        x[t, t] = 1
        Wr[4 * t:4 * t + 4, t] = torch.tensor([1.0, 2.0, 3.0, 4.0], device="cuda").bfloat16()
    ids = _check(lib, (x, Wr, Wg, Wu, Wd), 4)[1]
    assert torch.equal(ids, (4 * torch.arange(8, device="cuda")[:, None] + torch.arange(3, -1, -1, device="cuda")).int())


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_kinds_and_fp32_routers(lib, act, normalize):
    for dtype in (BF16, F16):
        _check(lib, _inputs(6, 136, 48, 10, dtype, 2, router=F32), 3, act, normalize)


def test_many_slots_of_one_expert(lib):
    # groups of sixteen, the last one of one slot
    x, Wr, Wg, Wu, Wd = _inputs(33, 72, 40, 4, BF16, 3)
    x = x.abs()
    Wr[:] = 0
    Wr[2] = 1
    y, ids, weights = _check(lib, (x, Wr, Wg, Wu, Wd), 2)
    assert bool((ids == torch.tensor([2, 0], device="cuda", dtype=torch.int32)).all())   # ties: the lowest index


def test_ties_and_signs_of_zero(lib):
    x, Wr, Wg, Wu, Wd = _inputs(5, 64, 16, 200, BF16, 4)
    Wr[:] = 0
    Wr[150] = -0.0
    assert bool((lib.moe_route(x, Wr, 7)[0] == torch.arange(7, device="cuda")).all())
    Wr[:] = torch.randn(10, 64, device="cuda").bfloat16().repeat(20, 1)   # every logit twenty times
    _check(lib, (x, Wr, Wg, Wu, Wd), 30, normalize=False)


def test_given_choices(lib):
    # twice the same expert, outside the experts, weights of any sign, a token without an expert
    x, _, Wg, Wu, Wd = _inputs(6, 96, 40, 5, F16, 5)
    ids = torch.tensor([[0, 0, 1], [4, -1, 3], [5, 7, -9], [2, 2, 2], [1 << 30, 0, 4], [-(1 << 31), 3, 1]], dtype=torch.int32, device="cuda")
    weights = torch.tensor([[0.5, 0.25, -2.0], [1, 1, 1], [1, 1, 1], [0, 0, 1], [3, -1, 0.125], [1, 0, 1e-3]], device="cuda")
    y = lib.moe_experts(x, ids, weights, Wg, Wu, Wd)
    _check_experts(lib, y, x, ids, weights, Wg, Wu, Wd, "silu")
    assert not y[2].any()
    out = torch.full_like(x, 7.0)
    assert lib.moe_experts(x[:0], ids[:0], weights[:0], Wg, Wu, Wd).shape == (0, 96)
    assert lib.moe_experts(x, ids, weights, Wg, Wu, Wd, out=out) is out and torch.equal(out, y)


def test_values_that_are_not_finite(lib):
    x, Wr, Wg, Wu, Wd = _inputs(20, 128, 64, 8, BF16, 6)
    y, ids, weights = lib.moe(x, Wr, Wg, Wu, Wd, 3, routing=True)
    bad = x.clone()
    bad[3, 5] = float("nan")
    bad[7, 0] = float("inf")
    yb, ib, wb = lib.moe(bad, Wr, Wg, Wu, Wd, 3, routing=True)
    keep = [t for t in range(20) if t not in (3, 7)]
    assert torch.equal(y[keep], yb[keep]) and torch.equal(ids[keep], ib[keep])
    assert torch.isnan(yb[3]).all() and bool((ib[3] == torch.arange(3, device="cuda")).all())
    assert bool(((ib >= 0) & (ib < 8)).all()) and not torch.isfinite(yb[7]).any()
    # an expert that no token takes may hold anything
    used = torch.unique(ids)
    unused = [e for e in range(8) if e not in used.tolist()]
    few = lib.moe_experts(x[:1], ids[:1], weights[:1], Wg, Wu, Wd)
    for w in (Wg, Wu, Wd):
        for e in range(8):
            if e not in ids[0].tolist():
                w[e] = float("nan")
    assert torch.equal(lib.moe_experts(x[:1], ids[:1], weights[:1], Wg, Wu, Wd), few)


def test_router_logits_that_are_not_finite(lib):
    x = torch.ones(1, 8, device="cuda").bfloat16()
    Wr = torch.zeros(6, 8, device="cuda").bfloat16()
    Wr[:, 0] = torch.tensor([1.0, float("nan"), 3.0, -float("inf"), 2.0, float("nan")])
    ids, weights = lib.moe_route(x, Wr, 6)
    assert ids[0].tolist() == [2, 4, 0, 3, 1, 5]
    ids, weights = lib.moe_route(x, Wr, 4)
    want = np.exp(np.array([3.0, 2.0, 1.0, -np.inf]) - 3)
    assert ids[0].tolist() == [2, 4, 0, 3] and np.allclose(_host(weights)[0], want / want.sum(), rtol=1e-7)
    assert torch.isnan(lib.moe_route(x, Wr, 2, normalize=False)[1]).all()


def test_fp16_hidden_values_past_their_range(lib):
    # h beyond 65504, and one far below it in another slot: both leave y in range
    x, Wr, Wg, Wu, Wd = _inputs(4, 64, 48, 3, F16, 7)
    x[0] *= 300
    x[1] *= 2.0 ** -9
    Wg, Wu = Wg * 8, Wu * 8
    Wd = Wd * 2.0 ** -7
    ids = torch.tensor([[0, 1]] * 4, dtype=torch.int32, device="cuda")
    weights = torch.full((4, 2), 2.0 ** -3, device="cuda")
    y = lib.moe_experts(x, ids, weights, Wg, Wu, Wd)
    h = (x[0].double() @ Wg[0].double().t()).clamp(min=0) * (x[0].double() @ Wu[0].double().t())
    assert float(h.abs().max()) > 1e5 and bool(torch.isfinite(y).all())
    _check_experts(lib, y, x, ids, weights, Wg, Wu, Wd, "silu")


@pytest.mark.parametrize("tokens", [1, 9])
@pytest.mark.parametrize("cols,rows", [(64, 40), (65, 33), (127, 129), (333, 72), (200, 201)])
def test_strides_and_alignment(lib, tokens, cols, rows):
    # gate and up as halves of one tensor or apart by any number of entries; what lies around is NaN
    def inside(t, first, pad, gap):
        n = t.shape[0] if t.dim() == 3 else 1
        m, k = t.shape[-2:]
        buf = torch.full((first + n * (m * (k + pad) + gap) + 8,), float("nan"), dtype=t.dtype, device="cuda")
        v = torch.as_strided(buf, t.shape, ((m * (k + pad) + gap),) * (t.dim() - 2) + (k + pad, 1), first)
        v.copy_(t)
        return v
    for dtype in (BF16, F16):
        x, Wr, Wg, Wu, Wd = _inputs(tokens, cols, rows, 5, dtype, cols + tokens)
        both = torch.cat([Wg, Wu], 1)
        y = _check(lib, (x, Wr, both[:, :rows], both[:, rows:], Wd), 2)[0]
        for pad, gap in ((0, 0), (3, 5), (8, 64)):
            ops = inside(x, 1, pad, 0), inside(Wr, 3, pad, 0), inside(Wg, 1, pad, gap), inside(Wu, 6, pad, gap), inside(Wd, 5, pad, gap)
            got = _check(lib, ops, 2)[0]
            assert torch.allclose(got.float(), y.float(), rtol=2 ** -6, atol=1e-2)
        # rows of the experts one after the other: an expert's rows lie between the others'
        turned = [w.transpose(0, 1).contiguous().transpose(0, 1) for w in (Wg, Wu, Wd)]
        _check(lib, (x, Wr, *turned), 2)


def test_leading_dimensions(lib):
    x, Wr, Wg, Wu, Wd = _inputs(12, 64, 32, 4, BF16, 1)
    y, ids, weights = lib.moe(x, Wr, Wg, Wu, Wd, 2, routing=True)
    a, b, c = lib.moe(x.view(3, 4, 64), Wr, Wg, Wu, Wd, 2, routing=True)
    assert a.shape == (3, 4, 64) and b.shape == c.shape == (3, 4, 2)
    assert torch.equal(a.view(12, 64), y) and torch.equal(b.view(12, 2), ids) and torch.equal(c.view(12, 2), weights)
    assert torch.equal(lib.moe_experts(x.view(3, 4, 64), b, c, Wg, Wu, Wd), a)
    one = lib.moe(x[0], Wr, Wg, Wu, Wd, 2)
    assert one.shape == (64,) and torch.equal(one, y[0])


def test_a_token_alone_and_among_others(lib):
    # the choice is the same to the bit; y by different orders of its sums, each within the bound
    x, Wr, Wg, Wu, Wd = _inputs(50, 256, 72, 16, BF16, 9)
    y, ids, weights = lib.moe(x, Wr, Wg, Wu, Wd, 4, routing=True)
    for t in (0, 17, 49):
        a, b, c = lib.moe(x[t:t + 1], Wr, Wg, Wu, Wd, 4, routing=True)
        assert torch.equal(b[0], ids[t]) and torch.equal(c[0], weights[t])
        _check_experts(lib, a, x[t:t + 1], b, c, Wg, Wu, Wd, "silu")
    again = [lib.moe(x, Wr, Wg, Wu, Wd, 4) for _ in range(3)]
    assert all(torch.equal(z, y) for z in again)


def test_workspace(lib):
    x, Wr, Wg, Wu, Wd = _inputs(9, 136, 72, 12, F16, 8)
    y, ids, weights = lib.moe(x, Wr, Wg, Wu, Wd, 3, routing=True)
    need = lib.moe_workspace_bytes(9, 136, 72, 12, 3)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(2):   # what the first call left is no harm to the second
        assert torch.equal(lib.moe(x, Wr, Wg, Wu, Wd, 3, workspace=ws[:need]), y) and bool((ws[need:] == 0xFF).all())
    assert torch.equal(lib.moe_experts(x, ids, weights, Wg, Wu, Wd, workspace=ws[:need]), y)
    small = lib.moe_workspace_bytes(9, 136, 0, 12, 3)
    assert small <= need and torch.equal(lib.moe_route(x, Wr, 3, workspace=ws[:small])[0], ids)
    for bad in (lambda: lib.moe(x, Wr, Wg, Wu, Wd, 3, workspace=ws[:need - 256]), lambda: lib.moe_route(x, Wr, 3, workspace=ws[:small - 1]),
                lambda: lib.moe(x, Wr, Wg, Wu, Wd, 3, workspace=ws[1:])):
        with pytest.raises(lib.ExterndError):
            bad()


def test_side_stream(lib):
    x, Wr, Wg, Wu, Wd = _inputs(9, 136, 72, 12, BF16, 8)
    y = lib.moe(x, Wr, Wg, Wu, Wd, 3)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:   # two calls at once
        with torch.cuda.stream(s):
            late = torch.zeros_like(x)
            late.copy_(x)
            got.append(lib.moe(late, Wr, Wg, Wu, Wd, 3))
    torch.cuda.synchronize()
    assert all(torch.equal(z, y) for z in got)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("tokens", [1, 20])
def test_in_a_graph(lib, tokens, dtype):
    x, Wr, Wg, Wu, Wd = _inputs(tokens, 136, 72, 12, dtype, 8)
    lib.moe(x, Wr, Wg, Wu, Wd, 3)
    torch.cuda.synchronize()
    static = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, ids, weights = lib.moe(static, Wr, Wg, Wu, Wd, 3, routing=True)
    for k in range(4):
        new = _inputs(tokens, 136, 72, 12, dtype, 30 + k)[0] * 2.0 ** (2 * k - 4)
        static.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        want = lib.moe(new, Wr, Wg, Wu, Wd, 3, routing=True)
        assert all(torch.equal(a, b) for a, b in zip((y, ids, weights), want)), k


def test_refusals(lib):
    x, Wr, Wg, Wu, Wd = _inputs(4, 64, 32, 6, BF16, 0)
    ids, weights = lib.moe_route(x, Wr, 2)
    for bad in (lambda: lib.moe(x.float(), Wr, Wg, Wu, Wd, 2), lambda: lib.moe(x, Wr.half(), Wg, Wu, Wd, 2),
                lambda: lib.moe(x, Wr, Wg.half(), Wu, Wd, 2), lambda: lib.moe(x, Wr, Wg, Wu, Wd.cpu(), 2),
                lambda: lib.moe_experts(x, ids.long(), weights, Wg, Wu, Wd), lambda: lib.moe_experts(x, ids, weights.half(), Wg, Wu, Wd),
                lambda: lib.moe_route(x.float(), Wr, 2)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: lib.moe(x, Wr[:5], Wg, Wu, Wd, 2), lambda: lib.moe(x, Wr, Wg, Wu[:, :31], Wd, 2),
                lambda: lib.moe(x, Wr, Wg, Wu, Wd.transpose(1, 2), 2), lambda: lib.moe(x[:, :60], Wr, Wg, Wu, Wd, 2),
                lambda: lib.moe(x, Wr, Wg, Wu, Wd, 2, "relu"), lambda: lib.moe_experts(x, ids[:3], weights[:3], Wg, Wu, Wd),
                lambda: lib.moe_experts(x, ids, weights[:, :1], Wg, Wu, Wd), lambda: lib.moe(x, Wr, Wg[0], Wu[0], Wd[0], 2),
                lambda: lib.moe(x, Wr, Wg, Wu, Wd.transpose(1, 2).contiguous().transpose(1, 2), 2),
                lambda: lib.moe(x, Wr, Wg[:1].expand(6, 32, 64), Wu[:1].expand(6, 32, 64), Wd, 2),
                lambda: lib.moe(x, Wr, Wg, torch.cat([Wu, Wu], 1)[:, :32], Wd, 2)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lib.moe(x, Wr, Wg, Wu, Wd, 7), lambda: lib.moe(x, Wr, Wg, Wu, Wd, 0), lambda: lib.moe_route(x, Wr, 7),
                lambda: lib.moe_route(torch.zeros(4097, 64, device="cuda").bfloat16(), Wr, 2),
                lambda: lib.moe_route(x, torch.zeros(1025, 64, device="cuda").bfloat16(), 2)):
        with pytest.raises(lib.ExterndError):
            bad()
    with pytest.raises(lib.ExterndError, match="overlaps"):
        lib.moe(x, Wr, Wg, Wu, Wd, 2, out=x)
    leaf = x.clone().requires_grad_()
    for y in (lib.moe(leaf, Wr, Wg, Wu, Wd, 2), lib.moe_experts(leaf, ids, weights, Wg, Wu, Wd), lib.moe_route(leaf, Wr, 2)[1]):
        with pytest.raises(RuntimeError, match="has no gradient"):
            y.float().sum().backward()
    with torch.no_grad():
        assert torch.equal(lib.moe(leaf, Wr, Wg, Wu, Wd, 2), lib.moe(x, Wr, Wg, Wu, Wd, 2))
