"""CPU checks of how the gated block's products are run (csrc/gated_plan.hpp, host code): the shapes
that the GPU tests take reach every form, and a plan keeps what the kernels assume."""
import os
import shutil
import subprocess

import pytest

from gated_shapes import SHAPES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUS = 256   # MI355X

PROGRAM = r"""
#include <cstdio>
#include "gated_plan.hpp"
using namespace externd;
int main() {
  long long t, c, r, cus;
  while (scanf("%lld %lld %lld %lld", &t, &c, &r, &cus) == 4) {
    const GatedPlan f = plan_of(kFwd, t, r, steps_of(padded(c, 8)), cus), x = plan_dx(t, c, r, cus), w = plan_dw(t, c, r, cus);
    printf("%d %lld 1 %lld  ", f.kind, (long long)f.splits, (long long)steps_of(padded(c, 8)));
    printf("%d %lld %lld %lld  ", x.kind, (long long)x.splits, (long long)x.stacked, (long long)((x.stacked == 2 ? 2 : 4) * steps_of(r)));
    printf("%d %lld 1 %lld\n", w.kind, (long long)w.splits, (long long)(2 * steps_of(t)));
  }
}
"""
BIG, PAIR, DEEP = range(3)


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """plans(shapes) -> per shape the (kind, splits, stacked, steps) of the forward, dx and dW."""
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no host compiler")
    where = tmp_path_factory.mktemp("plan")
    (where / "plan.cpp").write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-I", os.path.join(ROOT, "ternary_rank_weight_amd", "csrc"), "-o", str(where / "plan"),
                    str(where / "plan.cpp")], check=True)

    def run(shapes, cus=CUS):
        text = "".join(f"{t} {c} {r} {cus}\n" for t, c, r in shapes)
        out = subprocess.run([str(where / "plan")], input=text, capture_output=True, text=True, check=True).stdout
        rows = [list(map(int, line.split())) for line in out.splitlines()]
        return [[tuple(row[i:i + 4]) for i in (0, 4, 8)] for row in rows]
    return run


def _counts(splits, steps):
    """Steps of a workgroup's unit: of the first splits and of the last."""
    whole = max(1, steps)
    per = -(-whole // splits)
    used = -(-whole // per)
    return used, {per, whole - (used - 1) * per}


def test_shapes_reach_every_form(plans):
    seen = set()
    for products in plans(SHAPES):
        for product, (kind, splits, stacked, steps) in enumerate(products):
            used, counts = _counts(splits, steps)
            for n in counts:
                if n >= 8:
                    seen.add((product, kind, used > 1, n % (4 if kind == DEEP else 6)))
    want = {(0, BIG, False): range(6), (0, PAIR, False): range(6), (0, DEEP, False): range(4), (0, DEEP, True): range(4),
            # dx has four segments and dW two, so that unsplit they take even numbers of steps
            (1, BIG, False): (0, 2, 4), (1, BIG, True): (0, 2, 3, 4, 5), (1, PAIR, False): (0, 2, 4), (1, DEEP, False): (0,),
            (1, DEEP, True): range(4),
            (2, BIG, False): (0, 2, 4), (2, PAIR, False): (0, 2, 4), (2, DEEP, False): (0, 2), (2, DEEP, True): range(4)}
    missing = [(form, n) for form, ns in want.items() for n in ns if (*form, n) not in seen]
    assert not missing


def test_plans_keep_what_the_kernels_assume(plans):
    shapes = [(t, c, r) for t in (1, 16, 33, 64, 65, 200, 777, 4096, 100000) for c in (1, 63, 64, 520, 2560, 9728, 40000)
              for r in (1, 65, 640, 4100, 9728, 1 << 21)]
    for cus in (256, 304, 32):
        for (t, c, r), products in zip(shapes, plans(shapes, cus)):
            for product, (kind, splits, stacked, steps) in enumerate(products):
                assert 1 <= splits <= 16 and (splits == 1 or steps >= 4 * splits)
                # the split forms that are instantiated
                assert splits == 1 or kind == DEEP or (kind == BIG and product == 1)
                assert stacked == 1 or (product == 1 and kind == DEEP and t <= 64)
                if kind == DEEP:
                    m, n = ((t, r), (stacked * t, c), (r, c))[product]
                    tiles = -(-m // 128) * -(-n // (64 if product == 0 else 128)) * (2 if product == 2 else 1)
                    assert tiles * splits <= cus
