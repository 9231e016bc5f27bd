"""GPU checks of what the 4-bit and gated operators refuse: outputs and workspaces that overlap
their inputs."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_outputs_on_inputs_are_refused(lib):
    W = torch.randn(64, 64, device="cuda")
    q = lib.q4_quantize(W)
    x = torch.randn(8, 64, device="cuda")
    keep = x.clone()
    with pytest.raises(lib.ExterndError, match="overlaps"):
        lib.q4_apply(q, x, out=x)
    with pytest.raises(lib.ExterndError, match="overlaps"):
        lib.q4_gated(q, q, x, out=x)
    ws = torch.empty((lib.q4_workspace_bytes(64, 8, torch.float32) + 256,), dtype=torch.uint8, device="cuda")
    y = ws[:8 * 64 * 4].view(torch.float32).view(8, 64)
    with pytest.raises(lib.ExterndError, match="overlaps"):
        lib.q4_apply(q, x, out=y, workspace=ws)
    h = torch.randn(8, 64, device="cuda").bfloat16()
    with pytest.raises(lib.ExterndError, match="overlaps"):
        lib.gated_forward(h, W.bfloat16(), W.bfloat16(), out=h)
    assert torch.equal(x, keep)
    # apart: rows of one buffer
    both = torch.randn(16, 64, device="cuda")
    assert torch.equal(lib.q4_apply(q, both[:8], out=both[8:]), lib.q4_apply(q, both[:8].clone()))
