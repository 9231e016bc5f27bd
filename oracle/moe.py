"""Plain fp64 mixture-of-experts layer."""
import numpy as np

from .gated import act


def route(x, Wr, top, normalize):
    """(ids, weights): largest logits first, the lower index of equal ones."""
    logits = x @ Wr.T
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :top]
    e = np.exp(logits - logits.max(1, keepdims=True))
    chosen = np.take_along_axis(e, ids, 1)
    return ids, chosen / (chosen if normalize else e).sum(1, keepdims=True)


def experts(x, ids, weights, Wg, Wu, Wd, name):
    """Weighted sum of the chosen experts; ids outside them add nothing."""
    y = np.zeros_like(x)
    for t in range(x.shape[0]):
        for e, w in zip(ids[t], weights[t]):
            if 0 <= e < Wg.shape[0]:
                y[t] += w * (Wd[e] @ (act(name, Wg[e] @ x[t])[0] * (Wu[e] @ x[t])))
    return y
