"""Parameters that are given other storage, sizes, strides or types between an AdamW object's steps."""
import pytest
import torch

import ternary_rank_weight_amd as trw

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture
def steps(monkeypatch):
    """AdamW on CPU tensors with the library's call replaced; the (address, entries, type) of each step's tensors."""
    seen = []

    def need(t, dtype, name):
        if t.dtype != dtype:
            raise TypeError(name)
        if not t.is_contiguous():
            raise ValueError(name)

    def step(table, count, opts, stream):
        seen.append([(t.param, t.grad, t.n, t.param_dtype) for t in table])
        return 0
    for name, value in (("_need", need), ("_op_device", lambda *t: -1), ("_current_device", lambda: -1),
                        ("_raw_stream", lambda index: 0), ("_adamw_step", step)):
        monkeypatch.setattr(trw, name, value)
    return seen


# the same address each time
CHANGES = {
    "shrunk": lambda p: p.data[:4],
    "one entry": lambda p: p.data[0, :1],
    "transposed": lambda p: p.data.t(),
    "strided": lambda p: p.data[:, ::2],
    "retyped": lambda p: p.data.view(F16),
    "as integers": lambda p: p.data.view(torch.int16),
    "narrower": lambda p: p.data.view(torch.uint8),
}


@pytest.mark.parametrize("change", CHANGES)
def test_another_shape_at_the_same_address_is_refused(steps, change):
    p, q = torch.nn.Parameter(torch.zeros(8, 8, dtype=BF16), requires_grad=False), torch.nn.Parameter(torch.zeros(5))
    opt = trw.AdamW([p, q])
    opt.step([torch.zeros_like(p), torch.zeros_like(q)])
    kept = p.data
    p.data = CHANGES[change](p)
    assert p.data_ptr() == kept.data_ptr()
    with pytest.raises((TypeError, ValueError)):
        opt.step([torch.zeros(p.shape, dtype=BF16), torch.zeros_like(q)])
    assert len(steps) == 1   # (the library was not called)
    p.data = kept
    opt.step([torch.zeros_like(p), torch.zeros_like(q)])
    assert steps[1][0][0] == kept.data_ptr() and steps[1][0][2:] == (64, 1) and steps[1][1][2:] == (5, 0)


def test_a_grown_parameter_is_refused(steps):
    whole = torch.zeros(16, 8)
    p = torch.nn.Parameter(whole[:8])
    opt = trw.AdamW([p])
    p.data = whole
    with pytest.raises(ValueError):
        opt.step([torch.zeros(16, 8)])
    assert not steps


def test_new_storage_and_another_view_of_all_entries(steps):
    p = torch.nn.Parameter(torch.zeros(8, 6, dtype=BF16))
    opt = trw.AdamW([p])
    p.data = torch.ones(8, 6, dtype=BF16)
    opt.step([torch.zeros_like(p)])
    assert steps[0][0][0] == p.data_ptr() and steps[0][0][2:] == (48, 1)
    p.data = p.data.view(4, 12)   # the same entries in the same order
    opt.step([torch.zeros(4, 12)])
    assert steps[1][0][0] == p.data_ptr() and steps[1][0][2:] == (48, 1)
    for other in (torch.ones(8, 7, dtype=BF16), torch.ones(8, 6), torch.ones(6, 8, dtype=BF16).t()):
        p.data = other
        with pytest.raises((TypeError, ValueError)):
            opt.step([torch.zeros(other.shape)])
    assert len(steps) == 2


def test_a_tensor_left_out_is_not_looked_at(steps):
    p = torch.nn.Parameter(torch.zeros(8, 8))
    opt = trw.AdamW([p, torch.zeros(3)])
    p.data = p.data[:4]
    opt.step([None, torch.zeros(3)])
    assert steps[0][0][2] == 0 and steps[0][1][2] == 3


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_steps_on_new_storage(lib, bits):
    w = torch.randn(40, 30, device="cuda")
    p, q = torch.nn.Parameter(w.clone()), w.clone()
    a, b = lib.AdamW([p], bits=bits), lib.AdamW([q], bits=bits)
    for k in range(3):
        g = torch.randn_like(w)
        a.step([g])
        b.step([g])
        assert torch.equal(p.detach(), q)
        old = p.data
        p.data = old.clone()
        old.fill_(7.0)   # (nothing writes here any more)
        assert p.data_ptr() != old.data_ptr()
    a.step([g])
    assert bool((old == 7.0).all())
    keep = p.data
    before = keep.clone()
    p.requires_grad_(False)   # (integers have no gradient)
    for change in (lambda t: t[:20], lambda t: t.t(), lambda t: t.view(torch.int32)):
        p.data = change(keep)
        with pytest.raises((TypeError, ValueError)):
            a.step([torch.zeros(p.shape, device="cuda")])
    assert torch.equal(keep, before)
