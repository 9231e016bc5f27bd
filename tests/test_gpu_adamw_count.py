"""GPU checks that an AdamW object has one count of steps for all of its tensors, as its documentation says: against the
oracle with that count, within the roundings that tests/test_gpu_adamw.py derives."""
import numpy as np
import pytest
import torch

from oracle import adamw as oa

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.mark.parametrize("bits", [8, 32])
def test_a_late_first_gradient_is_corrected_for_every_step(lib, bits):
    torch.manual_seed(bits)
    p, q = torch.randn(300, device="cuda"), torch.randn(70, device="cuda")
    opt = lib.AdamW([p, q], lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1, bits=bits)
    g = torch.randn(300, device="cuda")
    for _ in range(3):
        opt.step([g, None])
    w0, g = q.double().cpu().numpy(), (0.5 + torch.rand(70, device="cuda")) * torch.randn(70, device="cuda").sign()
    opt.step([None, g])
    m, v = oa.moments(np.zeros(70, np.float32), np.zeros(70, np.float32), g.cpu().numpy(), (0.9, 0.99))
    want, update = oa.weights(w0, m, v, 4, 1e-2, (0.9, 0.99), 1e-8, 0.1)
    assert np.all(np.abs(q.double().cpu().numpy() - want) <= 4 * E * np.abs(w0) + 12 * E * update)
    # 0.1 / (1 - 0.9^4) over the root of 0.01 / (1 - 0.99^4): 0.58 of lr, where a count of its own would give lr
    assert np.allclose(update, 1e-2 * 0.1 / (1 - 0.9 ** 4) / np.sqrt(0.01 / (1 - 0.99 ** 4)), rtol=1e-4)


def test_a_step_without_any_gradient_counts(lib):
    p = torch.randn(50, device="cuda")
    opt = lib.AdamW([p])
    before = p.clone()
    opt.step([None])
    opt.step()   # (no .grad either)
    assert torch.equal(p, before) and opt.state["step"][0] == 2 and not opt.state["m"].any()
