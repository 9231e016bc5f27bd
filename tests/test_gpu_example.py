"""The compressed MLP example runs end to end and its numbers make sense."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_compressed_mlp(lib):
    spec = importlib.util.spec_from_file_location("compressed_mlp", os.path.join(ROOT, "examples", "compressed_mlp.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    r = mod.run(hidden=1216, width=320, tokens=384, steps=6)
    assert 0 < r["h_4bit_tuned"] < r["h_4bit"] < 0.3
    assert r["energy_4bit"] > 0.98
    assert r["y_4bit"] < 0.3 and r["y_ternary"] < 0.6
