"""AdamW steps in numpy: moments by the 32-bit steps that define them (so that codes can be
compared bit by bit), weights in 64 bits; and the 8-bit codes by a search among their values."""
import numpy as np

BLOCK = 256
# values of the codes before the block's scale: 0 .. 126 of m (sign apart), 0 .. 247 of v
M_VALUES = np.array([k * 2.0 ** -9 if k < 8 else (8 + k % 8) * 2.0 ** (k // 8 - 10) for k in range(127)])
V_VALUES = np.array([k * 2.0 ** -17 if k < 8 else (8 + k % 8) * 2.0 ** (k // 8 - 18) for k in range(248)])
M_TOP, V_TOP = 134, 141


def blocks_of(x):
    """x filled up with zeros to whole blocks."""
    x = np.asarray(x).reshape(-1)
    return np.concatenate([x, np.zeros(-len(x) % BLOCK, x.dtype)]).reshape(-1, BLOCK)


def exponents(x):
    """Exponent bytes of float32 blocks."""
    a = np.where(np.isfinite(x), np.abs(x), np.float32(0)).max(1)
    return np.maximum(a.astype(np.float32).view(np.uint32) >> 23, 15).astype(np.uint8)


def _nearest(values, x):
    """Index of the nearest value, ties to the even index."""
    hi = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    up, down = values[hi] - x, x - values[hi - 1]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def encode_m(x):
    """(codes, exponents) of float32 moments in whole blocks."""
    b = exponents(x)
    scaled = np.abs(np.where(np.isfinite(x), x, 0).astype(np.float64)) * np.exp2(M_TOP - b.astype(np.float64))[:, None]
    code = _nearest(M_VALUES, scaled) + np.where(np.signbit(x), 128, 0)
    nan = ~np.isfinite(x)
    return np.where(nan, 0x7f, code).astype(np.uint8), b


def encode_v(x):
    b = exponents(x)
    scaled = np.where(np.isfinite(x), x, 0).astype(np.float64) * np.exp2(V_TOP - b.astype(np.float64))[:, None]
    code = _nearest(V_VALUES, scaled)
    code = np.where((code == 0) & (x > 0), 1, code)
    return np.where(np.isfinite(x), code, np.where(np.isnan(x), 0xff, 0xf8)).astype(np.uint8), b


def decode_m(code, b):
    value = np.append(M_VALUES, np.nan)[code & 127] * np.where(code > 127, -1.0, 1.0)
    return (value * np.exp2(b.astype(np.float64) - M_TOP)[:, None]).astype(np.float32)


def decode_v(code, b):
    value = np.concatenate([V_VALUES, [np.inf], np.full(7, np.nan)])[code]
    return (value * np.exp2(b.astype(np.float64) - V_TOP)[:, None]).astype(np.float32)


def moments(m, v, g, betas, grad_scale=1.0):
    """New fp32 moments."""
    f = np.float32
    with np.errstate(all="ignore"):
        g = g.astype(f) * f(grad_scale)
        m = f(betas[0]) * m + f(1.0 - betas[0]) * g
        v = f(betas[1]) * v + f(1.0 - betas[1]) * (g * g)
    return m, v


def weights(w, m, v, t, lr, betas, eps, decay):
    """New weights in 64 bits from this step's moments, and the size of the update."""
    with np.errstate(all="ignore"):
        m, v = m.astype(np.float64), v.astype(np.float64)
        update = lr / (1.0 - betas[0] ** t) * m / (np.sqrt(v / (1.0 - betas[1] ** t)) + eps)
        return w * (1.0 - lr * decay) - update, np.abs(update)
