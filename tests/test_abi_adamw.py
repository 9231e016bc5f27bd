"""C-ABI checks of the AdamW step that need no GPU: what it refuses before any HIP call.  (Addresses are
made up; nothing is read.)"""
import ctypes

import pytest
import torch

import ternary_rank_weight_amd as trw

# what is not refused ends at the missing device; with one it would run on these addresses
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the calls must not reach a GPU")

EINVAL = 1
G = 1 << 32


def tensor(at=1, n=1000, bits=32, param_dtype=1, grad_dtype=1, **other):
    """A tensor with its arrays 4 GB apart from `at` on."""
    t = trw._AdamTensor(at * G, (at + 1) * G, (at + 2) * G if param_dtype else None, (at + 3) * G, (at + 4) * G,
                        (at + 5) * G if bits == 8 else None, (at + 6) * G if bits == 8 else None, n, 0.1, param_dtype, grad_dtype, 0)
    for k, v in other.items():
        setattr(t, k, v)
    return t


def call(tensors, bits=32, step=100 * G, **other):
    o = trw._AdamOpts(1e-3, 0.9, 0.99, 1e-8, None, None, 1.0, bits, step)
    for k, v in other.items():
        setattr(o, k, v)
    table = (trw._AdamTensor * max(1, len(tensors)))(*tensors)
    return trw._adamw_step(table, len(tensors), o, None), trw._last_error().decode()


def refused(*a, **kw):
    status, text = call(*a, **kw)
    return status == EINVAL and text


def test_options():
    assert not refused([tensor()])
    for bad in ({"bits": 16}, {"beta1": 1.0}, {"beta2": -0.1}, {"beta1": float("nan")}, {"eps": -1e-9}, {"eps": float("inf")},
                {"lr": float("inf")}, {"step": None}, {"step": 100 * G + 4}, {"lr_device": 5 * G + 2}):
        assert refused([tensor()], **bad), bad
    assert not refused([tensor()], lr=float("inf"), lr_device=50 * G)
    assert trw._adamw_step(None, 1, trw._AdamOpts(), None) == EINVAL
    assert trw._adamw_step((trw._AdamTensor * 1)(tensor()), 1, None, None) == EINVAL
    assert trw._adamw_step((trw._AdamTensor * 1)(tensor()), -1, trw._AdamOpts(), None) == EINVAL


def test_tensors():
    for bad in ({"n": -1}, {"n": 1 << 41}, {"param_dtype": 3}, {"grad_dtype": -1}, {"param": None}, {"grad": None}, {"m": None},
                {"v": None}, {"decay": float("nan")}, {"param": G + 1}, {"grad": 2 * G + 1}, {"master": 3 * G + 4}, {"m": 4 * G + 8},
                {"v": 5 * G + 4}):
        assert refused([tensor(), tensor(10, **bad)]), bad
    assert refused([tensor(param_dtype=0, master=3 * G)])
    assert not refused([tensor(param_dtype=0)])
    assert not refused([tensor(n=0, param=None, grad=None)])
    assert refused([tensor(bits=8, m_exp=None)], bits=8) and refused([tensor(bits=8, v_exp=None)], bits=8)
    assert not refused([tensor(bits=8, m=4 * G + 4)], bits=8) and refused([tensor(bits=8, m=4 * G + 2)], bits=8)


def test_overlaps():
    # 1000 entries: 2000 bytes of parameters and gradients, 4096 of the rest; 8 bits: 1024 and 4
    a = dict(n=1000)
    assert "overlap" in refused([tensor(**a, grad=G)]) and "overlap" in refused([tensor(**a, grad=G + 1998)])
    assert not refused([tensor(**a, grad=G + 2000)])
    assert refused([tensor(**a, v=4 * G + 4080)]) and not refused([tensor(**a, v=4 * G + 4096)])
    assert refused([tensor(**a, master=4 * G - 16)]) and not refused([tensor(**a, master=4 * G - 4096)])
    assert refused([tensor(1, **a), tensor(10, **a, param=G + 4)]) and refused([tensor(1, **a), tensor(10, **a, grad=4 * G)])
    assert not refused([tensor(1, **a), tensor(10, **a, grad=2 * G)])   # two tensors may read one gradient
    assert refused([tensor(bits=8, m_exp=4 * G + 1023)], bits=8) and not refused([tensor(bits=8, m_exp=4 * G + 1024)], bits=8)
    assert refused([tensor()], step=G + 8) and refused([tensor()], lr_device=G + 4) and not refused([tensor()], lr_device=2 * G)
    assert refused([tensor()], grad_scale_device=100 * G + 28)
    # a long array over several short ones
    assert refused([tensor(1, n=8), tensor(10, n=8, grad=2 * G + 100), tensor(20, n=1 << 20, param=2 * G - 4096)])


def test_moments():
    call = lambda *p: trw._adamw_moments(*p[:4], 4, None, *p[4:])
    good = [G, 2 * G, 3 * G, 4 * G, 5 * G, 6 * G]
    assert call(*good) != EINVAL
    for i in range(6):
        assert call(*[None if j == i else p for j, p in enumerate(good)]) == EINVAL
        if i not in (1, 3):
            assert call(*[p + 2 if j == i else p for j, p in enumerate(good)]) == EINVAL
    assert call(*good[:4], G, 6 * G) == EINVAL and call(*good[:4], 5 * G, 5 * G + 4080) == EINVAL
    assert trw._adamw_moments(*good[:4], -1, None, *good[4:]) == EINVAL
    assert trw._adamw_moments(None, None, None, None, 0, None, None, None) == 0
