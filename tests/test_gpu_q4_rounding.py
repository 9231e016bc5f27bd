"""GPU checks of q4_reconstruct: each value is rounded once to the output's type, also where s c and m
are of very different size.  The references are exact: every s c + m here fits fp64."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _rounded(v, dtype):
    """Nearest value of the type, ties to even, straight from fp64."""
    bits, least, most = {torch.bfloat16: (8, -126, 3.3895313892515355e38), torch.float16: (11, -14, 65504.0),
                         torch.float32: (24, -126, 3.4028234663852886e38)}[dtype]
    e = np.maximum(np.frexp(v)[1], least + 1)
    q = np.ldexp(1.0, e - bits)
    r = np.rint(v / q) * q
    return np.where(np.abs(r) > most, np.copysign(np.inf, v), r)


def _check(lib, codes, s, m):
    group = 32
    back = lambda t: t.float().numpy().astype(np.float64).repeat(group, 1)[:, :codes.shape[1]]
    want = codes.numpy().astype(np.float64) * back(s) + back(m)
    q = lib.q4_pack(codes.cuda(), s.cuda(), m.cuda(), group)
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        got = lib.q4_reconstruct(q, dtype).double().cpu().numpy()
        wrong = got != _rounded(want, dtype)
        assert not wrong.any(), (dtype, int(wrong.sum()), want[wrong][:3], got[wrong][:3])


@pytest.mark.parametrize("cols", [256, 75])
def test_small_minima_beside_ties(lib, cols):
    # s c is a tie of bf16 or fp16 often, and m, far below fp32's last place, decides it
    gen = torch.Generator().manual_seed(cols)
    rows, groups = 512, -(-cols // 32)
    codes = torch.randint(0, 16, (rows, cols), generator=gen, dtype=torch.uint8)
    s = (torch.randint(128, 256, (rows, groups), generator=gen) / 128.0).bfloat16()
    sign = torch.randint(0, 2, (rows, groups), generator=gen) * 2 - 1
    m = (sign * torch.ldexp(torch.ones(rows, groups), -torch.randint(8, 41, (rows, groups), generator=gen))).bfloat16()
    _check(lib, codes, s, m)
    _check(lib, codes, s, -2 * s)          # both of one size
    _check(lib, codes, (s * 2.0 ** -20).bfloat16(), m)   # fp16's subnormal range


def test_ends_of_the_range(lib):
    # s c past fp32's largest number, the value not
    codes = torch.full((1, 32), 15, dtype=torch.uint8)
    codes[0, 1], codes[0, 2] = 14, 0
    s, m = (torch.tensor([[v]], dtype=torch.bfloat16) for v in (2.4e37, -1.6e38))
    _check(lib, codes, s, m)
    _check(lib, codes, s, 0 * m - 3e38)    # finite, and past the range on either side
    _check(lib, codes, -s, 0 * m - 2e38)
    _check(lib, codes, s / 2, 0 * m + 2e38)
