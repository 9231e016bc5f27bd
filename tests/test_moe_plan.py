"""CPU checks of how the experts' products are run (csrc/moe_plan.hpp, host code): the shapes that the GPU tests
take reach every form."""
import os
import shutil
import subprocess

import pytest

from moe_shapes import SHAPES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUS = 256   # MI355X

PROGRAM = r"""
#include <cstdio>
#include "moe_plan.hpp"
using namespace externd;
int main() {
  long long t, c, r, e, k, cus;
  while (scanf("%lld %lld %lld %lld %lld %lld", &t, &c, &r, &e, &k, &cus) == 6) {
    const MoeForms f = moe_forms(t, k, e, r, c, c, r, cus);
    printf("%d %d %d %d %d %d %d\n", moe_few(t, k, e), f.up, f.one, f.down, f.down_tiles, rows_apart_bits(c), rows_apart_bits(r));
  }
}
"""


@pytest.fixture(scope="module")
def forms(tmp_path_factory):
    """forms(shapes) -> per shape (choices in the first product, its waves a tile, one token's waves an expert, the second
    product's waves a tile, its tiles a wave, bits of how far apart a tile's rows are in either)."""
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no host compiler")
    where = tmp_path_factory.mktemp("plan")
    (where / "plan.cpp").write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-I", os.path.join(ROOT, "ternary_rank_weight_amd", "csrc"), "-o", str(where / "plan"),
                    str(where / "plan.cpp")], check=True)

    def run(shapes, cus=CUS):
        text = "".join("%d %d %d %d %d %d\n" % (*s[:5], cus) for s in shapes)
        out = subprocess.run([str(where / "plan")], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return run


def test_shapes_reach_every_form(forms):
    up, one, down, apart = set(), set(), set(), set()
    for (tokens, cols, rows, experts, top, alike), (few, waves, single, share, tiles, up_bits, down_bits) in zip(SHAPES, forms(SHAPES)):
        kind = "aligned" if alike and cols % 8 == 0 else "alike" if alike else "apart"
        up.add((few, waves, kind))
        up.add((0, waves, kind))   # (moe_experts on the same operands)
        if tokens == 1:
            one.add((rows % 8 == 0, single))
        else:
            down.add((rows % 8 == 0, share, tiles))
        apart |= {("up", up_bits), ("down", down_bits)}
    assert up >= {(few, waves, kind) for few in (0, 1) for waves in (4, 8, 16) for kind in ("aligned", "alike", "apart")}
    assert one >= {(al, sl) for al in (False, True) for sl in (1, 2, 4, 8, 16)}
    assert down >= {(al, sw, 1) for al in (False, True) for sw in (1, 2, 4, 8, 16)} | {(al, 1, 2) for al in (False, True)}
    assert apart == {(which, bits) for which in ("up", "down") for bits in range(4)}


def test_two_tiles_at_once_have_odd_ends(forms):
    # an odd number of the second product's groups of tiles, and rows past the last one's end
    ends = set()
    for (tokens, cols, rows, *_), (_, _, _, _, tiles, _, bits) in zip(SHAPES, forms(SHAPES)):
        if tiles == 2:
            groups = -(-cols // (16 << bits))
            ends.add((rows % 8 == 0, groups % 2, cols % 16 != 0))
    assert {(True, 1, True), (False, 1, True)} <= ends and (False, 0, True) in ends


def test_choice_of_forms(forms):
    # (the fewest waves that bring a launch to sixteen a compute unit; two tiles at once past twice that)
    for shape, (few, up, one, down, tiles, *_) in zip(SHAPES, forms(SHAPES)):
        tokens, cols, rows, experts, top, _ = shape
        assert few == (tokens <= 8 and tokens * top <= 64 and experts <= 256)
        assert (one > 0) == (tokens == 1) and (down > 0) == (tokens > 1)
        if tokens == 1:
            assert one * min(top, 16) <= 16 and up in (4, 8, 16)
    assert forms([(32, 2560, 768, 128, 8)])[0][:5] == (0, 4, 0, 1, 2)
    assert forms([(32, 2560, 768, 128, 8)], 2048)[0][3:5] == (2, 1)
