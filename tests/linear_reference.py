"""Operands of the linear layer and fp64 references on the device, each with the bound that is derived here.

Operands are 16-bit, products exact in fp32, sums fp32: a sum of n terms of total magnitude S is off by
at most (n + 64) 2^-24 S.  With |x||W|^T + |bias| = S, z is off by ez = (cols + 65) 2^-24 S.  An activation's
value moves by at most 1.13 of that and its slope by 0.9 (the Lipschitz constants), and they carry a few
fp32 roundings of their own, 16 and 32 of them.  y is rounded once: half a step u (2^-8 bf16, 2^-11 fp16).
dz is held in two parts of which the second is off by u of what the first is, u, so by u^2; its
smallest step is the type's subnormal one, for fp16 after the scaling that brings the row's largest to 2^14:
2^-25 / 2^14 of that.  Without an activation dz is dy.  Each gradient is rounded once."""
import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}
E = 2.0 ** -24


def inputs(tokens, cols, rows, dtype, seed, bias=True, residual=True):
    """x, W, bias, residual, dy."""
    rng = np.random.default_rng(seed)
    t = lambda *shape: torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda()
    x, W, b, r, dy = t(tokens, cols), 1.5 / np.sqrt(cols) * t(rows, cols), 0.5 * t(rows), t(tokens, rows), t(tokens, rows)
    x, W, b, r, dy = (v.to(dtype) for v in (x, W, b, r, dy))
    return x, W, b if bias else None, r if residual else None, dy


def _act(act, z):
    """act(z) and act'(z) in fp64 on the device (oracle/linear.py's formulas)."""
    if act is None:
        return z, torch.ones_like(z)
    if act == "silu":
        s = torch.special.expit(z)
        return z * s, s + z * s * (1 - s)
    if act == "gelu":
        phi = 0.5 * torch.special.erfc(-z / np.sqrt(2))
        return z * phi, phi + z * torch.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
    c = 2 * np.sqrt(2 / np.pi)
    a = c * (z + 0.044715 * z ** 3)
    s = torch.special.expit(a)
    return z * s, s + z * s * torch.special.expit(-a) * c * (1 + 3 * 0.044715 * z * z)


def _z(x, W, bias):
    X, V = x.double(), W.double()
    b = 0.0 if bias is None else bias.double()
    size = X.abs() @ V.abs().t() + (0.0 if bias is None else bias.double().abs())
    return X @ V.t() + b, (x.shape[1] + 65) * E * size


def forward_checks(x, W, bias, act, residual):
    """[(name, fp64 value, tolerance)] of z and y."""
    z, ez = _z(x, W, bias)
    a, _ = _act(act, z)
    r = torch.zeros_like(z) if residual is None else residual.double()
    y = a + r
    ea = ez if act is None else 1.13 * ez + 16 * E * z.abs()
    un = 1.02 * U[x.dtype]
    return [("z", z, ez + 1e-30), ("y", y, ea + 2 * E * (a.abs() + r.abs()) + un * y.abs() + TINY[x.dtype])]


def gradient_checks(x, W, bias, dy, act):
    """[(name, fp64 value, tolerance)] of dx, dW and db."""
    dtype, (tokens, cols), rows = x.dtype, x.shape, W.shape[0]
    X, V, D = x.double(), W.double(), dy.double()
    z, ez = _z(x, W, bias)
    _, slope = _act(act, z)
    dz = D * slope
    u = 1.02 * U[dtype]
    exact = D.abs() * (0.9 * ez + 32 * E * (1 + z.abs())) if act is not None else torch.zeros_like(dz)
    held = exact
    if act is not None:
        top = float(dz.abs().max()) if dz.numel() else 0.0
        held = exact + u * u * dz.abs() + (TINY[dtype] if dtype == torch.bfloat16 else top * 2.0 ** -38)
    m = dz.abs() + held
    dx, dw, db = dz @ V, dz.t() @ X, dz.sum(0)
    end = lambda want, tol: tol + u * (want.abs() + tol) + TINY[dtype]
    return [("dx", dx, end(dx, held @ V.abs() + (2 * rows + 128) * E * (m @ V.abs()))),
            ("dW", dw, end(dw, held.t() @ X.abs() + (2 * tokens + 128) * E * (m.t() @ X.abs()))),
            ("db", db, end(db, exact.sum(0) + (tokens + 64) * E * (dz.abs() + exact).sum(0)))]
