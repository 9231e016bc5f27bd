"""Pins of the plain 4-bit and gated-block oracles: hand-worked groups, the
layout's round trip, and gradients against central differences."""
import numpy as np
import pytest

from oracle import gated, q4


def test_symmetric_group_by_hand():
    # max|w| = 7 -> scale 1; ties to even, -8 is never reached from max|w| / 7
    w = np.zeros((1, 32), dtype=np.float32)
    w[0, :6] = [7, -7, 0.5, 1.5, -2.5, 3.4]
    codes, s, m = q4.quantize(w, 32, True)
    assert s.tolist() == [[1.0]] and m is None
    assert codes[0, :7].tolist() == [15, 1, 8, 10, 6, 11, 8]
    assert q4.values(codes, s, m, 32)[0, :6].tolist() == [7, -7, 0, 2, -2, 3]


def test_asymmetric_group_by_hand():
    # min -1, max 14 -> scale 1, minimum -1
    w = np.full((1, 3), -1, dtype=np.float32)
    w[0, 1:] = [14, 0.4]
    codes, s, m = q4.quantize(w, 64, False)
    assert s.tolist() == [[1.0]] and m.tolist() == [[-1.0]] and codes.tolist() == [[0, 15, 1]]
    assert q4.values(codes, s, m, 64).tolist() == [[-1, 14, 0]]


@pytest.mark.parametrize("symmetric", [True, False])
def test_constant_zero_and_bad_groups(symmetric):
    w = np.zeros((4, 64), dtype=np.float32)
    w[1] = 3.0
    w[2, 40] = np.inf
    w[3, 0] = np.nan
    codes, s, m = q4.quantize(w, 32, symmetric)
    v = q4.values(codes, s, m, 32)
    assert np.all(v[0] == 0)
    assert np.allclose(v[1], 3.0, rtol=2 ** -8)
    assert np.all(v[2, :32] == 0) and np.all(np.isnan(v[2, 32:]))
    assert np.all(np.isnan(v[3, :32])) and np.all(v[3, 32:] == 0)


@pytest.mark.parametrize("symmetric", [True, False])
def test_error_is_half_a_step(symmetric):
    w = np.random.default_rng(0).standard_normal((5, 300)).astype(np.float32)
    codes, s, m = q4.quantize(w, 64, symmetric)
    step = np.repeat(s, 64, axis=1)[:, :300]
    # the rounded scale (and minimum) move the ends by at most 15 2^-9 steps and 2^-9 |min|
    slack = 15 * 2.0 ** -8 * step + (0 if symmetric else 2.0 ** -8 * np.abs(np.repeat(m, 64, axis=1)[:, :300]))
    assert np.all(np.abs(q4.values(codes, s, m, 64) - w) <= 0.5 * step + slack)


def test_layout_words_by_hand():
    codes = np.zeros((17, 130), dtype=np.uint8)
    codes[0, 0], codes[0, 1], codes[0, 7] = 1, 2, 15
    codes[3, 8 * 2 + 32 * 3] = 9        # row 3, piece 2, word 3
    codes[16, 129] = 5                  # second tile, second chunk
    w = q4.pack_codes(codes)
    assert w.shape == (2, 2, 64, 4)
    assert w[0, 0, 0, 0] == 1 | 2 << 16 | 15 << 28
    assert w[0, 0, 3 + 32, 3] == 9
    assert w[1, 1, 0, 0] == 5 << 16
    assert np.count_nonzero(w) == 3


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_slopes_against_differences(name):
    g = np.linspace(-9, 9, 181)
    e = 1e-5
    diff = (gated.act(name, g + e)[0] - gated.act(name, g - e)[0]) / (2 * e)
    assert np.max(np.abs(diff - gated.act(name, g)[1])) <= 1e-9


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_gradients_against_differences(name):
    rng = np.random.default_rng(1)
    x, Wg, Wu = rng.standard_normal((3, 4)), rng.standard_normal((5, 4)), rng.standard_normal((5, 4))
    dh = rng.standard_normal((3, 5))
    grads = gated.backward(x, Wg, Wu, dh, name)
    e = 1e-6
    for k, grad in enumerate(grads):
        ops = [x, Wg, Wu]
        for i in np.ndindex(grad.shape):
            up, down = [o.copy() for o in ops], [o.copy() for o in ops]
            up[k][i] += e
            down[k][i] -= e
            diff = np.sum(dh * (gated.forward(*up, name)[0] - gated.forward(*down, name)[0])) / (2 * e)
            assert abs(diff - grad[i]) <= 1e-7 * (1 + abs(grad[i]))
