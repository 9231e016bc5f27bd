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


def linear(x=A, w=B, bias=None, residual=None, y=D, z=None, ldr=32, act=0, dtype=1, tokens=4, ws=None, wsb=0):
    return trw._linear_forward(x, tokens, 64, 64, w, 32, 64, bias, residual, ldr, dtype, act, None, y, z, ws, wsb)


def test_linear_forward():
    assert not refused(linear()) and not refused(linear(bias=C, residual=F, z=G)) and not refused(linear(residual=A, bias=B))
    assert refused(linear(y=A), "y", "x") and refused(linear(y=off(B, 32 * 128 - 2)), "w") and not refused(linear(y=off(B, 32 * 128)))
    assert refused(linear(bias=off(D, 254)), "bias") and not refused(linear(bias=off(D, 256)))
    assert refused(linear(residual=D), "residual") and not refused(linear(residual=off(D, 256), ldr=1 << 20)) and refused(linear(residual=off(D, 254), ldr=1 << 20))
    assert refused(linear(z=off(D, 252)), "z", "y") and refused(linear(z=A), "z", "x")
    bad = lambda **kw: linear(**kw) == EINVAL
    assert bad(act=4) and bad(act=-1) and bad(dtype=3) and bad(tokens=-1) and bad(residual=F, ldr=31) and bad(x=None) and bad(y=None)
    assert bad(x=off(A, 1)) and bad(z=off(G, 2)) and bad(bias=off(C, 1)) and linear(dtype=0) == 4 and linear(tokens=0) == 0


def linear_backward(z=D, dy=G, dx=None, dw=None, db=None, act=0, tokens=4, x=A):
    return trw._linear_backward(x, tokens, 64, 64, B, 32, 64, z, dy, 32, 1, act, None, dx, dw, db, None, 0)


def test_linear_backward():
    H = ctypes.c_void_p(9 << 32)
    assert not refused(linear_backward(dx=H, dw=C, db=F)) and not refused(linear_backward(act=3, dx=D))
    for at, name in ((A, "x"), (B, "w"), (D, "z"), (G, "dy")):
        assert refused(linear_backward(dx=at), "dx", name) and refused(linear_backward(dw=at), "dw", name)
        assert refused(linear_backward(db=at), "db", name)
    assert refused(linear_backward(dx=H, dw=off(H, 510)), "dw", "dx") and refused(linear_backward(dw=H, db=off(H, 4094)), "db", "dw")
    bad = lambda **kw: linear_backward(**kw) == EINVAL
    assert bad(dx=H, z=None) and bad(dx=H, dy=None) and bad(dx=H, x=None) and bad(act=5, dx=H) and not bad(dx=H, z=None, act=3)
    assert linear_backward() == 0 and linear_backward(tokens=0, dx=H) == 0
    assert trw._linear_forward_ws(0, 64, 32, 1) == 0 and trw._linear_backward_ws(4, 64, 32, 7, 1) == 0


H, I, J = (ctypes.c_void_p((k + 10) << 32) for k in range(3))


def experts(**kw):
    w = trw._MoeWeights(B, C, D, 6, 32, 64, 64, 2048, 32, 2048)
    for k, v in kw.items():
        setattr(w, k, v)
    return w


def moe(x=A, wr=F, y=G, ids=H, weights=I, top=2, tokens=4, dtype=1, wr_dtype=1, act=0, ws=None, wsb=0, ldx=64, ldr=64, **kw):
    return trw._moe(x, tokens, ldx, wr, ldr, wr_dtype, top, 1, ctypes.byref(experts(**kw)), dtype, act, None, y, ids, weights, ws, wsb)


def test_moe():
    # 6 experts of 32 x 64: 24576 bytes of each matrix; y 512 bytes, ids and weights 32
    assert not refused(moe()) and moe(tokens=0) == 0 and not refused(moe(wr_dtype=0)) and not refused(moe(wu=B.value))
    for at, name in ((A, "x"), (F, "wr"), (B, "wg"), (C, "wu"), (D, "wd")):
        assert refused(moe(y=at), "y", name) and refused(moe(ids=at), "ids", name) and refused(moe(weights=at), "weights", name)
        if at is not A and at is not F:
            assert refused(moe(y=off(at, 24574)), "y", name) and not refused(moe(y=off(at, 24576)))
    assert refused(moe(ids=off(G, 508)), "ids", "y") and not refused(moe(ids=off(G, 512)))
    assert refused(moe(weights=off(H, 28)), "weights", "ids")
    # between two experts that lie apart
    assert not refused(moe(y=off(B, 4096), up_stride=1 << 20)) and refused(moe(y=off(B, (1 << 21) + 2), up_stride=1 << 20))
    need = trw._moe_ws(4, 64, 32, 6, 2)
    assert refused(moe(ws=G, wsb=need), "workspace", "y") and refused(moe(ws=off(A, 256), wsb=need), "workspace", "x")
    assert not refused(moe(ws=J, wsb=need)) and trw._moe_ws(4, 64, 0, 6, 2) < need
    bad = lambda **kw: moe(**kw) == EINVAL
    assert bad(x=None) and bad(wr=None) and bad(y=None) and bad(ids=None) and bad(weights=None) and bad(wg=None) and bad(wd=None)
    assert bad(top=0) and bad(top=7) and bad(tokens=-1) and bad(act=3) and bad(dtype=5) and bad(wr_dtype=2) and bad(ldx=63) and bad(ldr=63)
    assert bad(up_ld=63) and bad(down_ld=31) and bad(up_stride=0) and bad(down_stride=-1) and bad(rows=0) and bad(experts=0)
    assert bad(x=off(A, 1)) and bad(ids=off(H, 2)) and bad(wu=C.value + 1) and bad(wr=off(F, 2), wr_dtype=0)
    unsupported = lambda **kw: moe(**kw) == 4
    assert unsupported(dtype=0) and unsupported(experts=1025) and unsupported(top=65, experts=100) and unsupported(tokens=4097)
    assert unsupported(cols=(1 << 21) + 64, up_ld=1 << 22, ldx=1 << 22, ldr=1 << 22)
    assert trw._moe_ws(0, 64, 32, 6, 2) == 0 and trw._moe_ws(4, 64, 32, 6, 7) == 0 and trw._moe_ws(4097, 64, 32, 6, 2) == 0


def test_moe_parts():
    route = lambda ids=H, weights=I, wr=F: trw._moe_route(A, 4, 64, 64, wr, 6, 64, 1, 1, 2, 1, None, ids, weights, None, 0)
    assert not refused(route()) and refused(route(ids=A), "ids", "x") and refused(route(weights=off(F, 764)), "weights", "wr")
    assert route(ids=None) == EINVAL and route(wr=None) == EINVAL
    given = lambda y=G, ids=H, weights=I: trw._moe_experts(A, 4, 64, ids, weights, 2, ctypes.byref(experts()), 1, 0, None, y, None, 0)
    assert not refused(given()) and not refused(given(ids=A)) and refused(given(y=H), "y", "ids") and refused(given(y=off(I, 30)), "y", "weights")
    assert given(ids=None) == EINVAL and given(weights=None) == EINVAL and given(y=None) == EINVAL
    assert trw._moe_experts(A, 4, 64, H, I, 2, None, 1, 0, None, G, None, 0) == EINVAL
