"""GPU checks of the 4-bit products' forms for matrices of many rows: eight-wave workgroups (512 row
tiles and more) over types, group sizes, kinds and token counts, and the staged copy of aligned x
(more than 16 tokens, 2^24 entries and more).  References in fp64 on the device; tolerances as
derived in tests/test_gpu_q4.py."""
import pytest
import torch

pytestmark = pytest.mark.gpu

HALF_ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}


def _matrix(lib, rows, cols, group, symmetric, seed):
    """(Q4, its fp64 values, the magnitudes that enter a sum per unit |x|)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 16, (rows, cols), generator=gen, device="cuda", dtype=torch.uint8)
    groups = -(-cols // group)
    s = (0.01 + 0.01 * torch.rand(rows, groups, generator=gen, device="cuda")).bfloat16()
    m = None if symmetric else (-0.1 * torch.rand(rows, groups, generator=gen, device="cuda")).bfloat16()
    wide = lambda t: t.double().repeat_interleave(group, 1)[:, :cols]
    c = codes.double()
    if symmetric:
        values, size = (c - 8) * wide(s), (c + 16 + 24) * wide(s)
    else:
        values, size = c * wide(s) + wide(m), (c + 16 + 16) * wide(s) + wide(m).abs()
    return lib.q4_pack(codes, s, m, group), values, size


def _x(tokens, cols, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    return torch.randn(tokens, cols, generator=gen, device="cuda").to(dtype)


def _check(lib, q, values, size, x):
    y = lib.q4_apply(q, x).double()
    X = x.double()
    want = X @ values.t()
    tol = (2 * q.cols + 128) * 2.0 ** -24 * (X.abs() @ size.t()) + HALF_ULP[x.dtype] * 1.01 * want.abs() + TINY[x.dtype]
    err = (y - want).abs() / tol
    assert bool((err <= 1).all()), (x.shape, float(err.max()))


@pytest.mark.parametrize("group,symmetric", [(32, True), (32, False), (64, True), (64, False), (128, True), (128, False)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_many_rows(lib, dtype, group, symmetric):
    for cols in (264, 203):
        q, values, size = _matrix(lib, 8203, cols, group, symmetric, group + cols)
        for tokens in (1, 4, 5, 16, 17, 33, 49, 70):
            _check(lib, q, values, size, _x(tokens, cols, dtype, tokens))


@pytest.mark.parametrize("group,symmetric", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_staged_copy_of_aligned_rows(lib, dtype, group, symmetric):
    rows, cols = 8200, 2056
    assert rows * cols >= 1 << 24
    q, values, size = _matrix(lib, rows, cols, group, symmetric, group)
    for tokens in (16, 17, 32, 48, 64, 81):
        _check(lib, q, values, size, _x(tokens, cols, dtype, tokens))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_gated_many_rows(lib, dtype):
    for group, symmetric, cols in ((32, False, 264), (128, True, 203)):
        qg, vg, sg = _matrix(lib, 8203, cols, group, symmetric, 1)
        qu, vu, su = _matrix(lib, 8203, cols, group, symmetric, 2)
        for tokens in (1, 5, 16, 17, 48, 65):
            x = _x(tokens, cols, dtype, tokens)
            X = x.double()
            g, u = X @ vg.t(), X @ vu.t()
            eg, eu = ((2 * cols + 128) * 2.0 ** -24 * (X.abs() @ s.t()) for s in (sg, su))
            a = g * torch.sigmoid(g)
            # the activation: slope at most 1.13, a few fp32 roundings of |g|
            ea = 1.13 * eg + 16 * 2.0 ** -24 * g.abs()
            tol = ea * (u.abs() + eu) + a.abs() * eu + HALF_ULP[dtype] * 1.02 * (a * u).abs() + TINY[dtype]
            assert bool(((lib.q4_gated(qg, qu, x).double() - a * u).abs() <= tol).all()), (tokens, cols)
