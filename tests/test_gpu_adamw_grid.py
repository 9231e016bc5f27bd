"""GPU checks of AdamW where a tensor has more pieces than workgroups are resident, in the kinds whose registers allow
different numbers of them: every entry has to be what it is in a small tensor, bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("dtype,grad,master", [(F32, F32, False), (BF16, F32, True), (F16, F32, True), (BF16, F32, False),
                                               (BF16, BF16, True), (F16, F16, False)])
def test_more_pieces_than_workgroups(lib, dtype, grad, master, bits):
    torch.manual_seed(0)
    n = 3 * 1024 * 4096 + 5 * 256 + 77   # (at most 1024 workgroups on 256 compute units, 4096 entries at a time)
    p, g = torch.randn(n, device="cuda").to(dtype), (0.1 * torch.randn(n, device="cuda")).to(grad)
    cuts = [0, 256, 4096 * 700, 4096 * 768, 4096 * 1024, 4096 * 2500 + 512, n - 77 - 256, n]
    parts = [p[a:b].clone() for a, b in zip(cuts, cuts[1:])]
    whole, apart = lib.AdamW([p], bits=bits, master=master), lib.AdamW(parts, bits=bits, master=master)
    for _ in range(2):
        whole.step([g])
        apart.step([g[a:b].clone() for a, b in zip(cuts, cuts[1:])])
    assert all(torch.equal(p[a:b], q) for a, b, q in zip(cuts, cuts[1:], parts))
    for x, y in zip(whole.moments(), apart.moments()):
        assert torch.equal(whole.piece(x, 0), torch.cat([apart.piece(y, i) for i in range(len(parts))]))
    assert torch.equal(whole.state["step"], apart.state["step"])


@pytest.mark.parametrize("dtype,grad,master", [(F32, BF16, False), (F16, F32, False), (BF16, F16, True)])
def test_a_first_call_that_is_captured(lib, dtype, grad, master):
    torch.manual_seed(1)
    p = torch.randn(5000, device="cuda").to(dtype)
    q = p.clone()
    g = torch.randn(5000, device="cuda").to(grad)
    a, b = lib.AdamW([p], master=master), lib.AdamW([q], master=master)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step([g])
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        b.step([g])
        assert torch.equal(p, q)
