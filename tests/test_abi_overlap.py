"""C-ABI checks that need no GPU: the 4-bit and gated operators refuse outputs that overlap what they
read or write besides, before any HIP call.  (Addresses are made up; nothing is read.)"""
import ctypes

import pytest
import torch

import ternary_rank_weight_amd as trw

# what is not refused ends at the missing device; with one it would run on these addresses
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the calls must not reach a GPU")

EINVAL = 1
A, B, C, D, F, G = (ctypes.c_void_p((k + 1) << 32) for k in range(6))   # 4 GB apart


def off(p, n):
    return ctypes.c_void_p(p.value + n)


def refused(status, *names):
    text = trw._last_error().decode()
    return status == EINVAL and "overlaps" in text and all(n in text for n in names)


def q4(rows, cols, group=32, codes=A, scales=B, mins=None):
    return trw._Q4(codes, scales, mins, rows, cols, group, 0)


def apply(w, x, tokens, ldx, y, dtype=0, ws=None, wsb=0):
    return trw._q4_apply(ctypes.byref(w), x, tokens, ldx, dtype, None, y, ws, wsb)


def test_apply():
    w = q4(32, 64)
    # 3 tokens of 64 floats, 100 apart: bytes 0-255, 400-655, 800-1055; the output has 3 * 32 * 4 = 384 bytes
    for at in (0, 255, 252, -380, 400, 1052, 700):
        assert refused(apply(w, C, 3, 100, off(C, at - at % 4)), "output", "x"), at
    for at in (-384, 1056, 5000):
        assert not refused(apply(w, C, 3, 100, off(C, at))), at
    # between two rows: 2 tokens, 1000 floats apart, output of 256 bytes
    assert not refused(apply(w, C, 2, 1000, off(C, 256)))
    assert not refused(apply(w, C, 2, 1000, off(C, 4000 - 256)))
    assert refused(apply(w, C, 2, 1000, off(C, 4000 - 252)))
    assert refused(apply(w, C, 2, 1000, off(C, 4000 + 252)))
    # the weights: 2 tiles of 1 chunk, 2048 bytes of codes, 256 of scales
    assert refused(apply(w, C, 1, 64, off(A, 2044)), "codes") and not refused(apply(w, C, 1, 64, off(A, 2048)))
    assert refused(apply(w, C, 1, 64, off(B, 252)), "scales") and not refused(apply(w, C, 1, 64, off(B, 256)))
    assert refused(apply(q4(32, 64, mins=D), C, 1, 64, off(D, 252)), "mins")
    # a workspace (6 fp32 tokens are staged) on the output, on x
    need = trw._q4_ws(64, 6, 0)
    assert refused(apply(w, C, 6, 64, D, 0, D, need), "workspace", "output")
    assert refused(apply(w, C, 6, 64, D, 0, off(C, 1280), need), "workspace", "x")
    assert not refused(apply(w, C, 6, 64, D, 0, F, need))
    assert not refused(apply(w, C, 1, 64, D, 0, D, need))   # not used: nothing is staged


def test_gated_4bit():
    g, u = q4(32, 64), q4(32, 64, codes=D, scales=F)
    call = lambda y, a=g, b=u: trw._q4_gated(ctypes.byref(a), ctypes.byref(b), C, 1, 64, 0, 0, None, y, None, 0)
    assert refused(call(off(D, 16)), "codes") and refused(call(F), "scales") and refused(call(A), "codes")
    assert not refused(call(G)) and not refused(call(G, g, g))


def test_quantize_pack_reconstruct():
    quantize = lambda W, codes, scales, mins: trw._q4_quantize(W, 32, 64, 64, 0, 32, None, codes, scales, mins)
    assert refused(quantize(A, off(A, 16), B, None), "codes", "W")
    assert refused(quantize(A, B, off(B, 2040), None), "scales", "codes")
    assert refused(quantize(A, B, C, C), "mins", "scales")
    assert not refused(quantize(A, off(A, 32 * 64 * 4), B, C))
    pack = lambda src, s, codes, scales: trw._q4_pack(src, s, None, 32, 64, 32, None, codes, scales, None)
    assert refused(pack(A, B, off(A, 16), D), "codes", "codes_in")
    assert refused(pack(A, B, C, off(B, 8)), "scales", "scales_in")
    assert not refused(pack(A, B, C, D))
    back = lambda out: trw._q4_reconstruct(ctypes.byref(q4(32, 64)), 0, None, out)
    assert refused(back(off(A, 2044)), "codes") and not refused(back(C))


def forward(x=A, wg=B, wu=C, h=D, g=None, u=None):
    return trw._gated_forward(x, 4, 64, 64, wg, wu, 32, 64, 1, 0, None, h, g, u, None, 0)


def test_gated_forward():
    assert not refused(forward()) and not refused(forward(wu=B)) and not refused(forward(g=F, u=G))
    assert refused(forward(h=A), "h", "x") and refused(forward(h=off(B, 32 * 128 - 2)), "wg")
    assert refused(forward(h=C), "wu") and not refused(forward(h=off(B, 32 * 128)))
    assert refused(forward(g=F, u=off(F, 508)), "u", "g") and not refused(forward(g=F, u=off(F, 512)))
    assert refused(forward(g=off(D, 252), u=F), "g", "h") and refused(forward(g=F, u=A), "u", "x")


def backward(dh=G, dx=None, dwg=None, dwu=None, g=D, u=F):
    return trw._gated_backward(A, 4, 64, 64, B, C, 32, 64, g, u, dh, 32, 1, 0, None, dx, dwg, dwu, None, 0)


def test_gated_backward():
    H = ctypes.c_void_p(9 << 32)
    assert not refused(backward(dx=H)) and not refused(backward(dx=H, u=D)) and not refused(backward(dwg=H, dwu=off(H, 4096)))
    for at, name in ((A, "x"), (B, "wg"), (C, "wu"), (D, "g"), (F, "u"), (G, "dh")):
        assert refused(backward(dx=at), "dx", name)
        assert refused(backward(dwg=H, dwu=at), "dwu", name)
    assert refused(backward(dwg=H, dwu=off(H, 4094)), "dwu", "dwg") and refused(backward(dx=H, dwg=H, dwu=A))
