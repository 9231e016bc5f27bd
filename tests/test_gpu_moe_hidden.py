"""GPU check that the experts keep every bit of an fp32 h between their products.

Exact integers: g and u are whole numbers of two 16-bit weights each, g at least 64, where silu(g) is g in fp32, and
h = g u is odd or even below 2^24, which fp32 holds and 23 bits do not.  An output is the difference of two such h, at most
100, so it is exact in 16 bits too: there is no tolerance."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


def _pairs(count, seed):
    """(g, u, g', u') with g u and g' u' in 2^23 .. 2^24 and 0 < g u - g' u' <= 100."""
    rng, out = random.Random(seed), []
    while len(out) < count:
        g, u = rng.randrange(2049, 4096, 2), rng.randrange(2049, 8192)
        if not 1 << 23 < g * u < 1 << 24:
            continue
        other = rng.randrange(1025, 8192, 2)
        r = g * u % other
        if 0 < r <= 100 and 64 <= g * u // other < 1 << 14 and g * u - r > 1 << 23:
            out.append((g, u, other, g * u // other))
    return out


def _weights(experts, cols, rows, dtype, seed):
    """Wg, Wu, Wd and y for x = 1, 1, 0, ..."""
    Wg, Wu = torch.zeros(2, experts, rows, cols, dtype=torch.float64)
    Wd, y = torch.zeros(experts, cols, rows, dtype=torch.float64), torch.zeros(experts, cols, dtype=torch.float64)
    for e in range(experts):
        for n, (g, u, g2, u2) in enumerate(_pairs(rows // 2, 100 * seed + e)):
            for W, k, v in ((Wg, 2 * n, g), (Wu, 2 * n, u), (Wg, 2 * n + 1, g2), (Wu, 2 * n + 1, u2)):
                W[e, k, 0], W[e, k, 1] = v // 128 * 128, v % 128
            Wd[e, n % cols, 2 * n], Wd[e, n % cols, 2 * n + 1] = 1, -1
            y[e, n % cols] = g * u - g2 * u2
    back = [w.to(dtype).cuda() for w in (Wg, Wu, Wd)]
    assert all(torch.equal(w.double().cpu(), v) for w, v in zip(back, (Wg, Wu, Wd)))   # (the type holds them)
    return (*back, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("cols,rows", [(64, 128), (67, 131), (200, 72)])
@pytest.mark.parametrize("tokens", [1, 5, 40])
def test_every_bit_of_h(lib, tokens, cols, rows, dtype):
    Wg, Wu, Wd, y = _weights(3, cols, rows, dtype, cols)
    x = torch.zeros(tokens, cols, dtype=dtype, device="cuda")
    x[:, :2] = 1
    ids = (torch.arange(tokens, device="cuda", dtype=torch.int32) % 3)[:, None].contiguous()
    got = lib.moe_experts(x, ids, torch.ones(tokens, 1, device="cuda"), Wg, Wu, Wd)
    assert torch.equal(got.double().cpu(), y[ids[:, 0].cpu().long()])
    Wr = torch.zeros(3, cols, dtype=dtype, device="cuda")   # (equal logits: the first)
    assert torch.equal(lib.moe(x, Wr, Wg, Wu, Wd, 1).double().cpu(), y[:1].expand(tokens, cols))
