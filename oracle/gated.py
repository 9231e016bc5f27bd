"""Plain fp64 gated feed-forward block, h = act(x Wg^T) * (x Wu^T), and its gradients."""
import numpy as np
from scipy.special import erfc, expit


def act(name, g):
    """(act(g), act'(g)) in fp64."""
    g = np.asarray(g, dtype=np.float64)
    if name == "silu":
        s = expit(g)
        return g * s, s + g * s * (1 - s)
    if name == "gelu":
        phi = 0.5 * erfc(-g / np.sqrt(2))
        return g * phi, phi + g * np.exp(-0.5 * g * g) / np.sqrt(2 * np.pi)
    if name == "gelu_tanh":
        # (1 + tanh(z)) / 2 = 1 / (1 + exp(-2 z)), which keeps its bits where tanh is near -1
        c = 2 * np.sqrt(2 / np.pi)
        z = c * (g + 0.044715 * g ** 3)
        return g * expit(z), expit(z) + g * expit(z) * expit(-z) * c * (1 + 3 * 0.044715 * g * g)
    raise ValueError(name)


def forward(x, Wg, Wu, name):
    """(h, g, u)."""
    g, u = x @ Wg.T, x @ Wu.T
    return act(name, g)[0] * u, g, u


def backward(x, Wg, Wu, dh, name):
    """(dx, dWg, dWu)."""
    g, u = x @ Wg.T, x @ Wu.T
    a, slope = act(name, g)
    dg, du = dh * u * slope, dh * a
    return dg @ Wg + du @ Wu, dg.T @ x, du.T @ x
