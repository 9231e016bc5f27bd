"""Operands of the gated block and fp64 references of its gradients on the device, with the bounds
that tests/test_gpu_gated_gradients.py derives."""
import numpy as np
import torch

from oracle import gated as og

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}
E = 2.0 ** -24


def inputs(tokens, cols, rows, dtype, seed):
    rng = np.random.default_rng(seed)
    t = lambda a: torch.from_numpy(a.astype(np.float32)).to(dtype).cuda()
    scale = 1.0 / np.sqrt(cols)
    return (t(rng.standard_normal((tokens, cols))), t(scale * 1.5 * rng.standard_normal((rows, cols))),
            t(scale * rng.standard_normal((rows, cols))), t(rng.standard_normal((tokens, rows))))


def references(x, wg, wu, dh, act, step=None):
    """[(name, fp64 gradient, tolerance before the output's rounding)].  step: the smallest difference of
    two dg or du that the parts hold (the subnormal step of dh's type by default)."""
    dtype, cols, tokens, rows = x.dtype, x.shape[1], x.shape[0], wg.shape[0]
    X, G, U_, D = (t.double() for t in (x, wg, wu, dh))
    gv, uv = X @ G.t(), X @ U_.t()
    a, slope = (torch.from_numpy(t).cuda() for t in og.act(act, gv.cpu().numpy()))
    eg, eu = (cols + 64) * E * (X.abs() @ G.abs().t()), (cols + 64) * E * (X.abs() @ U_.abs().t())
    ea, es = 1.13 * eg + 16 * E * gv.abs(), 0.9 * eg + 32 * E * (1 + gv.abs())
    un = U[dtype] * 1.02
    dg, du = D * uv * slope, D * a
    if step is None:
        step = TINY[dtype]
    edg = D.abs() * ((uv.abs() + eu) * es + eu * slope.abs()) + un ** 2 * dg.abs() + step
    edu = D.abs() * ea + un ** 2 * du.abs() + step
    mg, mu = dg.abs() + edg, du.abs() + edu
    return [("dx", dg @ G + du @ U_, edg @ G.abs() + edu @ U_.abs() + (4 * rows + 128) * E * (mg @ G.abs() + mu @ U_.abs())),
            ("dWg", dg.t() @ X, edg.t() @ X.abs() + (2 * tokens + 64) * E * (mg.t() @ X.abs())),
            ("dWu", du.t() @ X, edu.t() @ X.abs() + (2 * tokens + 64) * E * (mu.t() @ X.abs()))]
