"""The compressed MLP example leaves what it is given as it was."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_tune_leaves_the_weights_it_starts_from(lib):
    spec = importlib.util.spec_from_file_location("compressed_mlp", os.path.join(ROOT, "examples", "compressed_mlp.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, wg, wu = (torch.randn(n, 64, generator=gen, device="cuda") for n in (48, 96, 96))
    keep = wg.clone(), wu.clone()
    x = x.bfloat16()
    target = lib.gated_forward(x, wg.bfloat16(), wu.bfloat16())
    tg, tu = mod.tune(x, target, wg, wu, 32, 2, 0.005)
    assert torch.equal(wg, keep[0]) and torch.equal(wu, keep[1])
    assert not torch.equal(tg, wg) and not torch.equal(tu, wu)
