"""GPU checks of the linear layer, the experts and AdamW on operands of more than 2^31 entries: what lies behind is
compared with the same entries in small operands, or within the bounds of tests/linear_reference.py and
tests/test_gpu_moe.py."""
import pytest
import torch

from linear_reference import forward_checks, gradient_checks
from test_gpu_moe import _check_experts

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _memory():
    yield
    torch.cuda.empty_cache()


def _normal(scale, *shape):
    return torch.empty(shape, dtype=BF16, device="cuda").normal_(0, scale)


def _within(got, check):
    name, want, tol = check
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), (name, float((err / tol).max()))


@pytest.mark.parametrize("tokens", [2, 40])
@pytest.mark.parametrize("cols", [1032, 1033])
def test_linear(lib, tokens, cols):
    torch.manual_seed(0)
    rows, last = 1 << 21, slice((1 << 21) - 200, 1 << 21)
    W, x, b, r = _normal(0.03, rows, cols), _normal(1, tokens, cols), _normal(1, rows), _normal(1, tokens, rows)
    assert W.numel() > 1 << 31
    y, z = lib.linear_forward(x, W, b, "silu", r, save=True)
    checks = forward_checks(x, W[last], b[last], "silu", r[:, last])
    _within(z[:, last], checks[0])
    _within(y[:, last], checks[1])
    dy = _normal(1, tokens, rows)
    dw, db = lib.linear_backward(x, W, z, dy, "silu", need_dx=False)[1:]
    checks = gradient_checks(x, W[last], b[last], dy[:, last], "silu")
    _within(dw[last], checks[1])
    _within(db[last], checks[2])
    # dx: rows of W past 2^31 entries, the others' dy left out
    dy[:, :last.start] = 0
    dx = lib.linear_backward(x, W, z, dy, "silu", need_dw=False, need_db=False)[0]
    _within(dx, gradient_checks(x, W[last], b[last], dy[:, last], "silu")[0])


def test_experts(lib):
    torch.manual_seed(1)
    experts, rows, cols = 128, 4104, 4096
    Wg, Wu, Wd = _normal(0.02, experts, rows, cols), _normal(0.015, experts, rows, cols), _normal(0.015, experts, cols, rows)
    assert Wg.numel() > 1 << 31
    for tokens in (1, 3):
        x, weights = _normal(1, tokens, cols), torch.rand(tokens, 2, device="cuda")
        ids = torch.tensor([[127, 126], [125, 127], [0, 127]], dtype=torch.int32, device="cuda")[:tokens].contiguous()
        y = lib.moe_experts(x, ids, weights, Wg, Wu, Wd)
        used = sorted(set(ids.flatten().tolist()))
        few = torch.tensor([[used.index(e) for e in t] for t in ids.tolist()], dtype=torch.int32, device="cuda")
        _check_experts(lib, y, x, few, weights, Wg[used], Wu[used], Wd[used], "silu")
        assert torch.equal(y, lib.moe_experts(x, few, weights, Wg[used], Wu[used], Wd[used]))


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw(lib, bits):
    torch.manual_seed(2)
    n = (1 << 31) + 4 * 256 + 77
    p, g = _normal(1, n), _normal(0.01, n)
    end = (1 << 31) - 256   # (a block's start)
    pieces = [slice(0, 512), slice(end, n)]
    small = [p[s].clone() for s in pieces]
    opt, ref = lib.AdamW([p], bits=bits), lib.AdamW(small, bits=bits)
    for _ in range(2):
        opt.step([g])
        ref.step([g[s].clone() for s in pieces])
    assert all(torch.equal(p[s], q) for s, q in zip(pieces, small))
    if bits == 8:
        got, want = opt.moments(), ref.moments()
        for a, b in zip(got, want):
            assert torch.equal(a[pieces[1]], ref.piece(b, 1))
