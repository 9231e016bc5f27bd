"""GPU checks of the 4-bit products at the ends of x's range: the |x| of a group may add up to just
below 2^123.  Tolerance: as for any x, (2 cols + 128) 2^-24 of the sum of the terms' magnitudes (the
operand 16 + c, its offset, the minimum), and the output's rounding."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens", [1, 9, 20])
@pytest.mark.parametrize("group,symmetric", [(128, True), (128, False), (32, True)])
def test_group_sums_to_2_123(lib, dtype, tokens, group, symmetric):
    rows, cols = 40, 256
    gen = torch.Generator().manual_seed(tokens)
    codes = torch.randint(0, 16, (rows, cols), generator=gen, dtype=torch.uint8)
    s = (2.0 ** -60 * (1 + torch.rand(rows, cols // group, generator=gen))).bfloat16()
    m = None if symmetric else (-7.5 * s.float()).bfloat16()
    x = (2 * torch.rand(tokens, cols, generator=gen) - 1) * (2.0 ** 123 / group)
    x[0] = 0
    x[0, 5::group] = 2.0 ** 122.5   # and all of it in one entry
    x = x.to(dtype)
    q = lib.q4_pack(codes.cuda(), s.cuda(), None if m is None else m.cuda(), group)
    y = lib.q4_apply(q, x.cuda()).double().cpu().numpy()
    wide = lambda t: t.float().numpy().astype(np.float64).repeat(group, 1)
    c, xs = codes.numpy().astype(np.float64), x.double().numpy()
    w = (c - 8) * wide(s) if symmetric else c * wide(s) + wide(m)
    size = (c + 16 + (24 if symmetric else 16)) * wide(s) + (0 if symmetric else np.abs(wide(m)))
    want = xs @ w.T
    tol = (2 * cols + 128) * 2.0 ** -24 * (np.abs(xs) @ size.T)
    tol += {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}[dtype] * 1.01 * np.abs(want)
    assert np.all(np.abs(y - want) <= tol)


def test_infinite_and_nan_entries(lib):
    q = lib.q4_quantize(torch.randn(40, 256, device="cuda"))
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.randn(4, 256, device="cuda").to(dtype)
        x[1, 3], x[2, 200] = float("inf"), float("nan")
        y = lib.q4_apply(q, x)
        assert bool(torch.isnan(y[1:3]).all()) and bool(torch.isfinite(y[[0, 3]]).all())
