"""Plain fp64 linear layer, y = act(x W^T + bias) + residual, and its gradients."""
import numpy as np

from .gated import act as _act


def act(name, z):
    """(act(z), act'(z)); name None: z and 1."""
    z = np.asarray(z, dtype=np.float64)
    return (z, np.ones_like(z)) if name is None else _act(name, z)


def forward(x, W, bias, name, residual):
    """(y, z); bias and residual may be None."""
    z = x @ W.T + (0.0 if bias is None else bias)
    return act(name, z)[0] + (0.0 if residual is None else residual), z


def backward(x, W, bias, dy, name):
    """(dx, dW, db)."""
    dz = dy * act(name, forward(x, W, bias, name, None)[1])[1]
    return dz @ W, dz.T @ x, dz.sum(0)
