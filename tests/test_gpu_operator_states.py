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


def test_a_gradient_that_is_not_there_raises(lib):
    # the 4-bit products and gated_forward have no gradient: asked for one, they say so and do not leave it out
    W = torch.randn(64, 64, device="cuda")
    q = lib.q4_quantize(W)
    x = torch.randn(8, 64, device="cuda", requires_grad=True)
    half = W.bfloat16().requires_grad_()
    for y, what in ((lib.q4_apply(q, x), "q4_apply"), (lib.q4_gated(q, q, x), "q4_gated"),
                    (lib.gated_forward(x.detach().bfloat16(), half, half), "gated")):
        assert y.requires_grad
        with pytest.raises(RuntimeError, match=what):
            y.float().sum().backward()
        assert x.grad is None and half.grad is None
    with pytest.raises(RuntimeError, match="out"):
        lib.q4_apply(q, x, out=torch.empty(8, 64, device="cuda"))
    with torch.no_grad():
        y = lib.q4_apply(q, x)
        assert not y.requires_grad and torch.equal(y, lib.q4_apply(q, x.detach()))
        out = torch.empty(8, 64, device="cuda")
        assert lib.q4_apply(q, x, out=out) is out
    assert torch.equal(lib.q4_apply(q, x), y) and not lib.q4_apply(q, x.detach()).requires_grad
    # with save the caller takes the gradient by gated_backward
    h, g, u = lib.gated_forward(x.detach().bfloat16(), half, half, save=True)
    assert not h.requires_grad


def test_forward_workspace_covers_any_alignment(lib):
    for cols in (9728, 4096, 1024, 264):
        for rows in (300, 40, 2048):
            for tokens in (1, 16, 17, 32, 33, 64, 300):
                any_ = lib.gated_forward_workspace_bytes(tokens, cols, rows, aligned=False)
                assert any_ >= lib.gated_forward_workspace_bytes(tokens, cols, rows), (tokens, cols, rows)
                any_ = lib.gated_backward_workspace_bytes(tokens, cols, rows, aligned=False)
                assert any_ >= lib.gated_backward_workspace_bytes(tokens, cols, rows), (tokens, cols, rows)


@pytest.mark.parametrize("tokens,cols,rows,aligned", [(32, 9728, 300, True), (100, 4096, 72, True), (40, 203, 72, False),
                                                      (100, 4095, 72, False)])
def test_forward_in_a_caller_workspace(lib, tokens, cols, rows, aligned):
    # split sums, padded copies, both: with what was there before, just enough, and not enough
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    x, wg, wu = (torch.randn(n, cols, generator=gen, device="cuda").bfloat16() for n in (tokens, rows, rows))
    want = lib.gated_forward(x, wg, wu, save=True)
    need = lib.gated_forward_workspace_bytes(tokens, cols, rows, aligned)
    assert need > 0
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    got = lib.gated_forward(x, wg, wu, save=True, workspace=ws[:need])
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and bool((ws[need:] == 0xFF).all())
    with pytest.raises(lib.ExterndError):
        lib.gated_forward(x, wg, wu, workspace=ws[:min(need - 256, 256)])
