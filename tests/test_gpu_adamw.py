"""GPU checks of the AdamW step against oracle/adamw.py.

Moments are fp32 sums and products in a stated order, so they and their codes are compared
bit by bit.  A weight is (1 - lr decay) w - update: in fp32 the constants, the two products and the
difference are rounded, 2^-24 each, and the update by its root, quotient and constants, ten roundings of 2^-24 at
most.  What 16-bit parameters hold is that, rounded by half a step more."""
import numpy as np
import pytest
import torch

from oracle import adamw as oa

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U = {F32: 0.0, BF16: 2.0 ** -8, F16: 2.0 ** -11}
TINY = {F32: 0.0, BF16: 2.0 ** -134, F16: 2.0 ** -25}
E = 2.0 ** -24


def _np(t):
    return t.detach().double().cpu().numpy().reshape(-1)


class _Run:
    """Steps of an optimizer beside the oracle's."""

    def __init__(self, lib, sizes, dtype, grad, bits, master, seed, betas=(0.9, 0.95), eps=1e-8, decay=0.1, lr=1e-2, views=False):
        self.lib, self.bits, self.betas, self.eps, self.lr = lib, bits, betas, eps, lr
        self.rng = np.random.default_rng(seed)
        self.grad = grad
        self.decay = list(decay) if isinstance(decay, (list, tuple)) else [decay] * len(sizes)
        flat = torch.from_numpy(self.rng.standard_normal(sum(sizes) + 2).astype(np.float32)).to(dtype).cuda()
        self.flat = flat
        self.params = list(flat[1:-1].split(sizes)) if views else [t.clone() for t in flat[1:-1].split(sizes)]
        self.opt = lib.AdamW(self.params, lr=lr, betas=betas, eps=eps, weight_decay=decay, bits=bits, master=master)
        self.m = [np.zeros(p.numel(), np.float32) for p in self.params]
        self.v = [np.zeros(p.numel(), np.float32) for p in self.params]
        self.master = master and dtype != F32
        self.t = 0

    def grads(self, spread=3.0):
        out = []
        for p in self.params:
            g = self.rng.standard_normal(p.numel()) * 1e-2 * np.exp(spread * self.rng.standard_normal(p.numel()))
            out.append(torch.from_numpy(g.astype(np.float32)).to(self.grad).cuda().view(p.shape))
        return out

    def step(self, grads, scale=1.0):
        w0 = [_np(self.opt.piece(self.opt.state["master"], i)) if self.master else _np(p) for i, p in enumerate(self.params)]
        self.opt.step(grads, grad_scale=scale)
        self.t += 1
        got = self.opt.moments()
        for i, p in enumerate(self.params):
            if grads[i] is None or not p.numel():
                continue
            m, v = oa.moments(self.m[i], self.v[i], grads[i].float().cpu().numpy().reshape(-1), self.betas, scale)
            want, update = oa.weights(w0[i], m, v, self.t, self.lr, self.betas, self.eps, self.decay[i])
            if self.bits == 8:
                n = p.numel()
                m = oa.decode_m(*oa.encode_m(oa.blocks_of(m))).reshape(-1)[:n]
                v = oa.decode_v(*oa.encode_v(oa.blocks_of(v))).reshape(-1)[:n]
            self.m[i], self.v[i] = m, v
            for flat, mine in zip(got, (m, v)):
                assert np.array_equal(self.opt.piece(flat, i).cpu().numpy().reshape(-1), mine, equal_nan=True), i
            tol = 4 * E * np.abs(w0[i]) + 12 * E * update
            if self.master:
                w = self.opt.piece(self.opt.state["master"], i)
                assert np.all((np.abs(_np(w) - want) <= tol) | np.isnan(want)), i
                assert torch.equal(w.to(p.dtype).view(torch.int16), p.view(torch.int16).view(w.shape))
            u = U[p.dtype]
            ok = np.abs(_np(p) - want) <= tol * (1 + u) + u * np.abs(want) + TINY[p.dtype]
            assert np.all(ok | np.isnan(want)) and np.array_equal(np.isnan(_np(p)), np.isnan(want)), i
        return grads


SIZES = [1, 3, 255, 256, 257, 0, 513, 2047, 2048, 2049, 5000, 100003]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("grad", [F32, BF16, F16])
@pytest.mark.parametrize("dtype,master", [(F32, False), (BF16, False), (BF16, True), (F16, False), (F16, True)])
def test_steps(lib, dtype, master, grad, bits):
    for views in (False, True):   # pieces of one buffer: starts of any alignment
        run = _Run(lib, SIZES, dtype, grad, bits, master, 7, views=views)
        ends = run.flat[[0, -1]].clone()
        for _ in range(3):
            run.step(run.grads())
        assert torch.equal(run.flat[[0, -1]], ends)
        step = run.opt.state["step"].cpu().numpy()
        assert step[0] == 3 and step[3] == 0 and np.allclose(step[1:3], [0.9 ** 3, 0.95 ** 3], rtol=1e-14)


@pytest.mark.parametrize("bits", [8, 32])
def test_state_past_a_tensors_end_stays_zero(lib, bits):
    run = _Run(lib, [300, 5], BF16, BF16, bits, True, 3)
    for _ in range(2):
        run.step(run.grads())
    state = run.opt.state
    for flat in (*run.opt.moments(), state["master"]):
        assert not flat[300:512].any() and not flat[517:].any() and flat[:300].any()


def test_many_tensors_of_several_kinds(lib):
    # more than a launch takes, of three kinds in turn, a decay for each
    rng = np.random.default_rng(0)
    params = [torch.from_numpy(rng.standard_normal(40 + i).astype(np.float32)).to((F32, BF16, F16)[i % 3]).cuda() for i in range(170)]
    decay = [0.01 * i for i in range(170)]
    opt = lib.AdamW(params, lr=0.1, betas=(0.5, 0.5), eps=1e-6, weight_decay=decay, bits=8)
    for t in (1, 2):
        w0 = [_np(p) for p in params]
        opt.step([torch.ones_like(p) for p in params])
        for i, p in enumerate(params):
            # every gradient is 1, and so is each corrected moment; m and v of 0.5 and 0.75 have codes
            want = w0[i] * (1 - 0.1 * decay[i]) - 0.1 / (1 + 1e-6)
            u = U[p.dtype]
            assert np.all(np.abs(_np(p) - want) <= 16 * E * (np.abs(w0[i]) + 1) + u * np.abs(want)), (t, i)
    assert opt.state["step"][0] == 2


def test_gradients_left_out_and_attribute_grads(lib):
    run = _Run(lib, [500, 600, 700], F32, F32, 32, False, 5)
    grads = run.grads()
    run.step(grads)
    before = run.params[1].clone()
    grads = run.grads()
    grads[1] = None
    run.step(grads)
    assert torch.equal(run.params[1], before)
    grads = run.grads()
    for p, g in zip(run.params, grads):
        p.grad = g
    twin = lib.AdamW([p.clone() for p in run.params], lr=run.lr, betas=run.betas, weight_decay=0.1,
                     state={k: None if v is None else v.clone() for k, v in run.opt.state.items()})
    twin.step(grads)
    run.opt.step()
    for p, q in zip(run.params, twin._params):
        assert torch.equal(p, q)


@pytest.mark.parametrize("bits", [8, 32])
def test_scaled_gradients_and_device_numbers(lib, bits):
    run = _Run(lib, [1000], BF16, F16, bits, True, 8)
    run.step(run.grads(1.0), scale=2.0 ** -5)
    run.step(run.grads(1.0), scale=0.37)
    a, b = (_Run(lib, [1000], F32, F32, bits, False, 9) for _ in range(2))
    grads = a.grads()
    a.opt.step(grads, lr=0.25, grad_scale=0.5)
    b.opt.step(grads, lr=torch.tensor([0.25], device="cuda"), grad_scale=torch.tensor(0.5, device="cuda"))
    assert torch.equal(a.params[0], b.params[0])


def test_values_that_are_not_finite(lib):
    for bits in (8, 32):
        run = _Run(lib, [1024], F32, F32, bits, False, 4)
        run.step(run.grads())
        grads = run.grads()
        grads[0][3], grads[0][300], grads[0][700], grads[0][701] = float("nan"), float("inf"), -float("inf"), 2e19
        with np.errstate(all="ignore"):
            run.step(grads)
        p = run.params[0]
        bad = ~torch.isfinite(p)
        assert bad[3] and bad[300] and bad[700] and int(bad.sum()) <= 4
        run.step(run.grads())
        assert bool((~torch.isfinite(run.params[0])).eq(bad).all())


def test_codes_over_their_whole_range(lib):
    # moments of every exponent: subnormal codes, ties, the largest and smallest block exponents
    rng = np.random.default_rng(1)
    for top in (-140, -126, -112, -100, -20, 0, 60, 126):
        size = np.exp2(top - 40.0 * rng.random(4096))
        size[::7] = np.exp2(np.round(np.log2(size[::7]))) * rng.integers(8, 16, size[::7].shape) / 8
        size[::5] *= 1 + 2.0 ** -4   # halfway between two codes
        size[::31] = 0.0
        x = (size * rng.choice([-1.0, 1.0], 4096)).astype(np.float32)
        p = torch.zeros(4096, device="cuda")
        opt = lib.AdamW([p], lr=0.0, betas=(0.0, 0.0), eps=1.0, weight_decay=0.0, bits=8)
        opt.step([torch.from_numpy(x).cuda()])
        m, v = oa.moments(np.float32(0), np.float32(0), x, (0.0, 0.0))
        for name, (code, b) in (("m", oa.encode_m(oa.blocks_of(m))), ("v", oa.encode_v(oa.blocks_of(v)))):
            got = opt.state[name].cpu().numpy()
            assert np.array_equal(got[4096:], b), (top, name)
            same = got[:4096] == code.reshape(-1)
            same |= (got[:4096] & 127 == 0) & (code.reshape(-1) & 127 == 0) if name == "m" else False   # a zero's sign
            assert same.all(), (top, name, np.flatnonzero(~same)[:5])
        gm, gv = opt.moments()
        assert np.array_equal(np.abs(gm.cpu().numpy()), np.abs(oa.decode_m(*oa.encode_m(oa.blocks_of(m))).reshape(-1)), equal_nan=True)
        assert np.array_equal(gv.cpu().numpy(), oa.decode_v(*oa.encode_v(oa.blocks_of(v))).reshape(-1), equal_nan=True)


def test_eight_bits_follow_thirty_two(lib):
    # a step by 8-bit moments is off by a code's half step of m (2^-4) and of v's root (2^-5), a little more
    # over steps that decay; entries near 0 by the subnormal step of their block
    a = _Run(lib, [65536], F32, F32, 32, False, 11, betas=(0.9, 0.99))
    b = _Run(lib, [65536], F32, F32, 8, False, 11, betas=(0.9, 0.99))
    start = a.params[0].clone()
    for _ in range(10):
        grads = a.grads(1.0)
        a.opt.step(grads)
        b.opt.step(grads)
    moved, apart = (a.params[0] - start).norm(), (a.params[0] - b.params[0]).norm()
    assert apart < 0.1 * moved


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_steps_count(lib, bits):
    a = _Run(lib, [3000, 70], BF16, BF16, bits, True, 13)
    b = _Run(lib, [3000, 70], BF16, BF16, bits, True, 13)
    grads = a.grads()
    lr = torch.tensor([1e-2], device="cuda")
    a.opt.step(grads, lr=lr)
    b.opt.step(grads, lr=1e-2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.opt.step(grads, lr=lr)
    for k in range(4):
        lr.fill_(1e-2 * (k + 1))
        for g in grads:
            g.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        b.opt.step(grads, lr=lr)
        for p, q in zip(a.params, b.params):
            assert torch.equal(p, q), k
        assert torch.equal(a.opt.state["step"], b.opt.state["step"])
        assert torch.equal(a.opt.state["m"], b.opt.state["m"]) and torch.equal(a.opt.state["v"], b.opt.state["v"])


def test_another_stream_and_repeated_runs(lib):
    results = []
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()):
        run = _Run(lib, [300000, 17], BF16, F32, 8, False, 21)
        grads = run.grads()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            for _ in range(3):
                run.opt.step(grads)
        torch.cuda.synchronize()
        results.append([p.clone() for p in run.params] + [run.opt.state["m"], run.opt.state["v"]])
    for other in results[1:]:
        assert all(torch.equal(x, y) for x, y in zip(results[0], other))


def test_state_of_a_stopped_run(lib):
    a = _Run(lib, [999, 2000], F16, F16, 8, True, 31)
    grads = [a.grads() for _ in range(4)]
    for g in grads[:2]:
        a.opt.step(g)
    params = [p.clone() for p in a.params]
    state = {k: v.clone() for k, v in a.opt.state.items()}
    b = lib.AdamW(params, lr=a.lr, betas=a.betas, eps=a.eps, weight_decay=0.1, bits=8, master=True, state=state)
    for g in grads[2:]:
        a.opt.step(g)
        b.step(g)
    for p, q in zip(a.params, params):
        assert torch.equal(p, q)


def test_a_saved_parameter_that_a_step_changes_is_noticed(lib):
    w = torch.randn(64, 64, device="cuda", requires_grad=True)
    x = torch.randn(3, 64, device="cuda", requires_grad=True)
    y = (x @ w).sum()
    lib.AdamW([w]).step([torch.ones_like(w)])
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        y.backward()


def test_refusals(lib):
    p, q = torch.zeros(64, device="cuda"), torch.zeros(64, 2, device="cuda", dtype=BF16)
    with pytest.raises(ValueError):
        lib.AdamW([])
    with pytest.raises(ValueError):
        lib.AdamW([p], bits=16)
    with pytest.raises(TypeError):
        lib.AdamW([p.double()])
    with pytest.raises(TypeError):
        lib.AdamW([p.cpu()])
    with pytest.raises(ValueError):
        lib.AdamW([q.t()])
    with pytest.raises(ValueError):
        lib.AdamW([p, q], weight_decay=[0.1])
    opt = lib.AdamW([p, q])
    with pytest.raises(ValueError):
        opt.step([p])
    with pytest.raises(ValueError):
        opt.step([torch.zeros(63, device="cuda"), torch.zeros_like(q)])
    with pytest.raises(TypeError):
        opt.step([torch.zeros_like(p).double(), torch.zeros_like(q)])
    with pytest.raises(ValueError):
        opt.step([torch.zeros(64), torch.zeros_like(q)])
    with pytest.raises(lib.ExterndError):   # the gradient is the parameter itself
        opt.step([p, torch.zeros_like(q)])
    with pytest.raises(lib.ExterndError):   # the same tensor twice
        lib.AdamW([p, p]).step([torch.ones_like(p), torch.ones_like(p)])
    with pytest.raises(lib.ExterndError):
        lib.AdamW([p], betas=(1.0, 0.9)).step([torch.ones_like(p)])
    with pytest.raises(lib.ExterndError):
        lib.AdamW([p]).step([torch.ones_like(p)], lr=float("nan"))
    with pytest.raises(ValueError):
        lib.AdamW([p]).step([torch.ones_like(p)], lr=torch.zeros(2, device="cuda"))
    state = lib.AdamW([p]).state
    with pytest.raises(ValueError):
        lib.AdamW([p], master=True, state=state)
    with pytest.raises(ValueError):
        lib.AdamW([torch.zeros(300, device="cuda")], state=state)
    with pytest.raises(TypeError):
        lib.AdamW([p], bits=8, state=state)
    assert not p.any() and not q.any()
