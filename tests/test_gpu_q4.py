"""GPU checks of the 4-bit group weights (quantize, pack, reconstruct, apply,
gated) against oracle/q4.py in fp64.

Tolerances.  Quantized words, tables and fp32 values are exact.  A product's
sums are fp32: at most cols + 64 additions of terms whose magnitudes add up to
S = sum |x| (|operand| s + |offset x| ...), the operand 16 + c (at most 31) and
its offset (24, or 16 and the minimum); each addition and product rounds by 2^-24
of a partial sum <= S (doubled for products), so |y - y64| <= (2 cols + 128) 2^-24 S +
u |y64|, u the output type's half ulp (2^-8 bf16, 2^-11 fp16, 2^-24 fp32; fp16
adds 2^-25 below its normal range).  The gated form multiplies two such sums
through an activation of slope at most 1.13."""
import numpy as np
import pytest
import torch

from oracle import gated as og
from oracle import q4 as oq

pytestmark = pytest.mark.gpu

HALF_ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}


def _host(t):
    return t.detach().cpu().double().numpy()


def _bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def _weights(rows, cols, seed):
    rng = np.random.default_rng(seed)
    return (0.02 * rng.standard_t(5, size=(rows, cols))).astype(np.float32)


def _make(lib, rows, cols, group, symmetric, seed):
    W = _weights(rows, cols, seed)
    codes, s, m = oq.quantize(W, group, symmetric)
    dev = lambda a, **k: None if a is None else torch.from_numpy(a).cuda().to(**k)
    q = lib.q4_pack(torch.from_numpy(codes).cuda(), dev(s, dtype=torch.bfloat16), dev(m, dtype=torch.bfloat16), group)
    return q, codes, s, m, oq.values(codes, s, m, group)


def _spread(codes, s, m, group):
    """Sum of term magnitudes per unit |x|: the operand's and its offset's, times the scale, and the minimum."""
    cols = codes.shape[1]
    sp = lambda t: np.repeat(np.abs(t.astype(np.float64)), group, axis=1)[:, :cols]
    if m is None:
        return (codes + 16.0 + 24.0) * sp(s)
    return (codes + 16.0 + 16.0) * sp(s) + sp(m)


def _x(tokens, cols, dtype, seed):
    rng = np.random.default_rng(seed + 1)
    return torch.from_numpy(rng.standard_normal((tokens, cols)).astype(np.float32)).to(dtype).cuda()


def _bound(x, spread, cols):
    return (2 * cols + 128) * 2.0 ** -24 * (np.abs(_host(x)) @ spread.T)


def _check_apply(lib, q, x, values, spread):
    y = lib.q4_apply(q, x)
    ref = _host(x) @ values.T
    tol = _bound(x, spread, q.cols) + HALF_ULP[x.dtype] * np.abs(ref) * 1.01 + TINY[x.dtype]
    err = np.abs(_host(y).reshape(ref.shape) - ref)
    assert np.all(err <= tol), float((err / tol).max())
    return y


SHAPES = [(1, 1), (16, 128), (17, 129), (5, 31), (33, 300), (100, 257), (48, 1000), (515, 640), (1040, 4100)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_quantize_is_exact(lib, group, symmetric, dtype):
    for rows, cols in [(1, 1), (16, 128), (17, 129), (33, 300), (5, 31), (40, 1000)]:
        W = torch.from_numpy(_weights(rows, cols, rows)).to(dtype)
        if rows == 33:
            W[3] = 0.0
            W[4, 10:200] = 0.25
            W[5, 40] = float("inf")
            W[6, 299] = float("nan")
            W[7] *= 1e-30 if dtype != torch.float16 else 1e-3
        codes, s, m = oq.quantize(W.float().numpy(), group, symmetric)
        q = lib.q4_quantize(W.cuda(), group, symmetric)
        v = lib.q4_reconstruct(q)
        want = oq.values(codes, s, m, group)
        with np.errstate(all="ignore"):
            want32 = want.astype(np.float32)
        assert np.array_equal(v.cpu().numpy(), want32, equal_nan=True), (rows, cols)
        got = q.codes.cpu().numpy().view(np.uint32).reshape(oq.pack_codes(codes).shape)
        full = oq.pack_codes(np.full((rows, cols), 15, np.uint8))   # compare the real entries only
        assert np.array_equal(got & full, oq.pack_codes(codes)), (rows, cols)
        table = q.scales.float().cpu().numpy().reshape(oq.pack_table(s, cols, group).shape)
        assert np.array_equal(table, oq.pack_table(s, cols, group), equal_nan=True)
        if not symmetric:
            table = q.mins.float().cpu().numpy().reshape(table.shape)
            assert np.array_equal(table, oq.pack_table(m, cols, group), equal_nan=True)
        for out in (torch.bfloat16, torch.float16):
            w16 = lib.q4_reconstruct(q, out).cpu()
            assert torch.equal(torch.nan_to_num(w16), torch.nan_to_num(torch.from_numpy(want32).to(out)))


def test_quantize_strided_and_misaligned(lib):
    W = torch.from_numpy(_weights(20, 333, 0)).cuda().to(torch.bfloat16)
    for view in (W[:, 1:300], W[3:, 7:], W[::2, :256]):
        a, b = lib.q4_quantize(view, 64, False), lib.q4_quantize(view.contiguous(), 64, False)
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales) and torch.equal(a.mins, b.mins)


@pytest.mark.parametrize("rows,cols", [(1, 1), (17, 129), (40, 300)])
@pytest.mark.parametrize("group", [32, 128])
def test_pack_layout(lib, rows, cols, group):
    rng = np.random.default_rng(rows)
    codes = rng.integers(0, 16, size=(rows, cols)).astype(np.uint8)
    s = rng.standard_normal((rows, -(-cols // group))).astype(np.float32)
    sb = torch.from_numpy(s).to(torch.bfloat16)
    q = lib.q4_pack(torch.from_numpy(codes).cuda(), sb.cuda(), (2 * sb).cuda(), group)
    words = oq.pack_codes(codes)
    assert np.array_equal(q.codes.cpu().numpy().view(np.uint32).reshape(words.shape), words)
    t = oq.pack_table(sb.float().numpy(), cols, group)
    assert np.array_equal(q.scales.float().cpu().numpy().reshape(t.shape), t)
    assert np.array_equal(q.mins.float().cpu().numpy().reshape(t.shape), 2 * t)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("group,symmetric", [(32, True), (32, False), (64, True), (64, False), (128, True), (128, False)])
def test_apply(lib, dtype, group, symmetric):
    for k, (rows, cols) in enumerate(SHAPES):
        q, codes, s, m, v = _make(lib, rows, cols, group, symmetric, k)
        spread = _spread(codes, s, m, group)
        for tokens in (1, 2, 5, 16, 17, 33, 64, 70)[k % 2::2]:
            _check_apply(lib, q, _x(tokens, cols, dtype, k), v, spread)


def test_apply_many_row_tiles(lib):
    # past 512 row tiles the waves hold two each: an odd last one
    q, codes, s, m, v = _make(lib, 16 * 600 + 3, 200, 32, True, 3)
    for tokens in (1, 20, 40):
        _check_apply(lib, q, _x(tokens, 200, torch.bfloat16, 3), v, _spread(codes, s, m, 32))


def test_apply_strides_and_shapes(lib):
    q, codes, s, m, v = _make(lib, 50, 264, 32, True, 1)
    spread = _spread(codes, s, m, 32)
    big = _x(12, 300, torch.bfloat16, 1)
    for x in (big[:, 8:272], big[:, 3:267], big[::3, :264], big[4, 5:269]):
        y = _check_apply(lib, q, x.reshape(-1, 264) if x.dim() == 1 else x, v, spread)
        assert torch.equal(lib.q4_apply(q, x), y.reshape(x.shape[:-1] + (50,)))
    x3 = big[:, :264].contiguous().view(3, 4, 264)
    assert lib.q4_apply(q, x3).shape == (3, 4, 50)
    assert torch.equal(lib.q4_apply(q, x3).view(12, 50), lib.q4_apply(q, x3.view(12, 264)))
    t = big[:, :264].t().contiguous().t()   # unit row stride
    assert torch.equal(lib.q4_apply(q, t), lib.q4_apply(q, t.contiguous()))
    e = big[:1, :264].expand(7, 264)
    assert torch.equal(lib.q4_apply(q, e), lib.q4_apply(q, e.contiguous()))
    assert lib.q4_apply(q, big[:0, :264]).shape == (0, 50)


def test_apply_repeats_and_token_independence(lib):
    q, *_ = _make(lib, 100, 700, 64, False, 2)
    x = _x(40, 700, torch.float32, 2)
    y = lib.q4_apply(q, x)
    assert torch.equal(y, lib.q4_apply(q, x))
    bad = x.clone()
    bad[7, 3] = float("nan")
    bad[21, 699] = float("inf")
    z = lib.q4_apply(q, bad)
    keep = [t for t in range(40) if t not in (7, 21)]
    assert torch.equal(z[keep], y[keep])
    assert torch.isnan(z[[7, 21]]).all()


def test_apply_bad_scale_stays_in_its_row(lib):
    W = _weights(40, 300, 5)
    W[11, 150] = np.nan
    q = lib.q4_quantize(torch.from_numpy(W).cuda(), 32, False)
    y = lib.q4_apply(q, _x(3, 300, torch.bfloat16, 5))
    assert torch.isnan(y[:, 11]).all() and torch.isfinite(y[:, [r for r in range(40) if r != 11]]).all()


def test_padding_codes_do_not_matter(lib):
    q, codes, *_ = _make(lib, 19, 200, 32, True, 6)
    x = _x(5, 200, torch.float16, 6)
    y = lib.q4_apply(q, x)
    pad = oq.pack_codes(np.full((19, 200), 15, np.uint8))
    noise = (~pad).view(np.int32).reshape(-1)   # 15 in every padding entry
    q2 = lib.Q4(q.codes | torch.from_numpy(noise).cuda(), q.scales, None, 19, 200, 32)
    assert torch.equal(lib.q4_apply(q2, x), y)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_out_and_workspace(lib, dtype):
    q, *_ = _make(lib, 64, 333, 32, True, 7)
    x = _x(9, 333, dtype, 7)
    y = lib.q4_apply(q, x)
    out = torch.full((9, 64), 7.0, dtype=dtype, device="cuda")
    need = lib.q4_workspace_bytes(333, 9, dtype)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    assert lib.q4_apply(q, x, out=out, workspace=ws) is out
    assert torch.equal(out, y)
    with pytest.raises(lib.ExterndError):
        lib.q4_apply(q, x, workspace=ws[:need // 2])


def test_apply_on_a_side_stream(lib):
    q, *_ = _make(lib, 512, 1024, 32, True, 8)
    x = _x(4, 1024, torch.float32, 8)
    want = lib.q4_apply(q, x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        late = torch.zeros_like(x)
        for _ in range(20):
            late = late + x / 20   # work that the product has to wait for
        late.copy_(x)
        got = lib.q4_apply(q, late)
    s.synchronize()
    assert torch.equal(got, want)


def test_apply_in_a_graph(lib):
    q, *_ = _make(lib, 512, 1024, 32, True, 9)
    xs = [_x(4, 1024, torch.bfloat16, k) for k in range(3)]
    x = xs[0].clone()
    lib.q4_apply(q, x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = lib.q4_apply(q, x)
    for _ in range(2):
        for v in xs:
            x.copy_(v)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, lib.q4_apply(q, v))


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_gated(lib, act, dtype):
    for k, (rows, cols, group, symmetric) in enumerate([(1, 1, 32, True), (33, 300, 64, False), (100, 257, 128, True),
                                                        (515, 640, 32, False), (48, 1000, 32, True)]):
        qg, *g, vg = _make(lib, rows, cols, group, symmetric, k)
        qu, *u, vu = _make(lib, rows, cols, group, symmetric, k + 50)
        for tokens in (1, 7, 16, 30, 65)[k % 2::2]:
            x = _x(tokens, cols, dtype, k)
            h = lib.q4_gated(qg, qu, x, act)
            xh = _host(x)
            gv, uv = xh @ vg.T, xh @ vu.T
            eg, eu = _bound(x, _spread(*g, group), cols), _bound(x, _spread(*u, group), cols)
            a = og.act(act, gv)[0]
            ref = a * uv
            # the activation's own fp32 steps: a few roundings of |g|
            ea = 1.13 * eg + 16 * 2.0 ** -24 * np.abs(gv)
            tol = ea * (np.abs(uv) + eu) + np.abs(a) * eu + HALF_ULP[dtype] * 1.02 * np.abs(ref) + TINY[dtype]
            err = np.abs(_host(h) - ref)
            assert np.all(err <= tol), (rows, cols, tokens, float((err / tol).max()))


def test_gated_in_wide_range(lib):
    # projections far out on both sides: h is 0 or g u, never NaN
    q, *_ = _make(lib, 32, 64, 32, True, 4)
    x = _x(3, 64, torch.float32, 4) * 1e4
    for act in ("silu", "gelu", "gelu_tanh"):
        h = lib.q4_gated(q, q, x, act)
        g = lib.q4_apply(q, x)
        assert torch.isfinite(h).all()
        far = g.abs() > 100
        assert far.any()
        want = torch.where(g > 0, g * g, torch.zeros_like(g))
        assert torch.allclose(h[far], want[far], rtol=1e-5)


def test_refusals(lib):
    q, *_ = _make(lib, 32, 64, 32, True, 0)
    qm, *_ = _make(lib, 32, 64, 32, False, 0)
    x = _x(2, 64, torch.float32, 0)
    with pytest.raises(TypeError):
        lib.q4_apply(q, x.double())
    with pytest.raises(TypeError):
        lib.q4_apply(q, x.cpu())
    with pytest.raises(ValueError):
        lib.q4_apply(q, x[:, :63])
    with pytest.raises(ValueError):
        lib.q4_apply(q, x, out=torch.empty(2, 31, device="cuda"))
    with pytest.raises(TypeError):
        lib.q4_apply(q, x, out=torch.empty(2, 32, device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError):
        lib.q4_gated(q, q, x, "relu")
    with pytest.raises(lib.ExterndError):
        lib.q4_gated(q, qm, x)
    with pytest.raises(ValueError):
        lib.q4_quantize(x, 48)
    with pytest.raises(TypeError):
        lib.q4_quantize(x.int(), 32)
    with pytest.raises(ValueError):
        lib.Q4(q.codes[:-4], q.scales, None, 32, 64, 32)
    with pytest.raises(ValueError):
        lib.Q4(q.codes, q.scales, None, 32, 64, 64)
    with pytest.raises(TypeError):
        lib.q4_pack(torch.zeros(4, 64, device="cuda"), q.scales, group=32)
    with pytest.raises(ValueError):
        lib.q4_pack(torch.zeros(4, 64, device="cuda", dtype=torch.uint8), q.scales, group=32)


def test_quantize_quotients_round_as_divisions(lib):
    # many scales and quotients at and next to ties: weights on coarse grids times odd scales
    rng = np.random.default_rng(11)
    W = (rng.integers(-255, 256, size=(512, 2048)) * rng.integers(128, 256, size=(512, 1)) * 2.0 ** -17).astype(np.float32)
    W[::2] = np.nextafter(W[::2], np.float32(np.inf)) * rng.uniform(0.5, 2, size=(256, 2048)).astype(np.float32)
    for symmetric in (True, False):
        codes, s, m = oq.quantize(W, 32, symmetric)
        v = lib.q4_reconstruct(lib.q4_quantize(torch.from_numpy(W).cuda(), 32, symmetric))
        assert np.array_equal(v.cpu().numpy(), oq.values(codes, s, m, 32).astype(np.float32))
