"""CPU checks of how the linear layer's products are run (csrc/linear_plan.hpp, host code): the shapes
that the GPU tests take reach every form, and a plan keeps what the kernels assume."""
import os
import shutil
import subprocess

import pytest

from linear_shapes import SHAPES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUS = 256   # MI355X

PROGRAM = r"""
#include <cstdio>
#include "linear_plan.hpp"
using namespace externd;
int main() {
  long long t, c, r, parts, cus;
  while (scanf("%lld %lld %lld %lld %lld", &t, &c, &r, &parts, &cus) == 5) {
    const GatedPlan f = plan_linear(kLin, t, r, steps_of(padded(c, 8)), cus), x = plan_linear_dx(t, c, r, parts, cus),
                    w = plan_linear_dw(t, c, r, parts, cus);
    printf("%d %lld 1 %lld  ", f.kind, (long long)f.splits, (long long)steps_of(padded(c, 8)));
    printf("%d %lld %lld %lld  ", x.kind, (long long)x.splits, (long long)x.stacked,
           (long long)((parts && x.stacked == 1 ? 2 : 1) * steps_of(r)));
    printf("%d %lld 1 %lld  ", w.kind, (long long)w.splits, (long long)((parts ? 2 : 1) * steps_of(t)));
    const LinearJoin j = linear_join(t, c, r, parts, cus);
    printf("%d %d %lld %lld %d\n", linear_takes_rows(t, c, r, true, cus), linear_takes_rows(t, c, r, false, cus), (long long)j.dx,
           (long long)j.dw, j.kind);
  }
}
"""
BIG, PAIR, DEEP, MID, SLIM = range(5)
TILES = {BIG: (256, 256), PAIR: (128, 128), DEEP: (128, 128), MID: (256, 192), SLIM: (128, 64)}
FAR = (DEEP, SLIM)


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """plans(shapes) -> per shape ([(kind, splits, stacked, steps) of the forward, dx and dW], few-token kernel when
    aligned, and when not, workgroups of dx and dW in one launch and their tiles)."""
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no host compiler")
    where = tmp_path_factory.mktemp("plan")
    (where / "plan.cpp").write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-I", os.path.join(ROOT, "ternary_rank_weight_amd", "csrc"), "-o", str(where / "plan"),
                    str(where / "plan.cpp")], check=True)

    def run(shapes, cus=CUS):
        text = "".join(f"{t} {c} {r} {int(parts)} {cus}\n" for t, c, r, parts in shapes)
        out = subprocess.run([str(where / "plan")], input=text, capture_output=True, text=True, check=True).stdout
        rows = [list(map(int, line.split())) for line in out.splitlines()]
        return [([tuple(row[i:i + 4]) for i in (0, 4, 8)], bool(row[12]), bool(row[13]), tuple(row[14:17])) for row in rows]
    return run


def counts(splits, steps):
    """Steps of a workgroup's unit: of the first splits and of the last."""
    whole = max(1, steps)
    per = -(-whole // splits)
    used = -(-whole // per)
    return used, {per, whole - (used - 1) * per}


def forms(entry):
    """(product, kind, split, steps modulo what its images repeat after) of units of eight steps and more."""
    products, rows = entry[:2]
    for product, (kind, splits, stacked, steps) in enumerate(products):
        used, ns = counts(splits, steps)
        if product == 0 and rows:
            continue
        for n in ns:
            if n >= 8:
                yield product, kind, used > 1, n % (4 if kind in FAR else 6)


WANT = {(product, kind, split, n) for product in range(3) for kind in TILES for split in (False, True) if not (split and kind == PAIR)
        for n in range(4 if kind in FAR else 6)}


def test_shapes_reach_every_form(plans):
    seen = {f for entry in plans(SHAPES) for f in forms(entry)}
    assert not WANT - seen


def test_shapes_reach_every_form_of_joined_gradients(plans):
    seen = {(product, joined[2], steps % (3 if joined[2] == SLIM else 6))
            for (t, c, r, parts), (products, _, _, joined) in zip(SHAPES, plans(SHAPES)) if joined[0]
            for product, steps in ((1, (2 if parts else 1) * (r // 64)), (2, (2 if parts else 1) * (t // 64))) if steps >= 8}
    want = {(product, kind, n) for product in (1, 2) for kind in (SLIM, MID) for n in range(3 if kind == SLIM else 6)}
    assert not want - seen


def test_plans_keep_what_the_kernels_assume(plans):
    shapes = [(t, c, r, parts) for t in (1, 16, 33, 64, 65, 200, 777, 4096, 100000) for c in (1, 63, 64, 520, 2560, 9728, 40000)
              for r in (1, 65, 640, 4100, 9728, 1 << 21) for parts in (False, True)]
    for cus in (256, 304, 32):
        for (t, c, r, parts), (products, rows, unaligned_rows, joined) in zip(shapes, plans(shapes, cus)):
            assert unaligned_rows == (t <= 32) and not (rows and t > 32) and (rows or t > 3)
            dx, dw, tiles = joined
            if dx:
                # as many workgroups as are resident, none without a tile
                tm, tn = TILES[tiles]
                most = [-(-m // tm) * -(-c // tn) for m in (t, r)]
                assert tiles in (SLIM, MID) and products[1][2] == 1 and 0 < dx <= most[0] and 0 < dw <= most[1]
                assert dx + dw <= (2 if tiles == SLIM else 1) * cus
            for product, (kind, splits, stacked, steps) in enumerate(products):
                assert 1 <= splits <= 16 and (splits == 1 or steps >= 4 * splits) and not (splits > 1 and kind == PAIR)
                assert stacked == 1 or (product == 1 and kind in FAR and t <= 64 and parts)
                if kind in FAR:
                    m, n = ((t, r), (stacked * t, c), (r, c))[product]
                    tm, tn = TILES[kind]
                    assert -(-m // tm) * -(-n // tn) * splits <= cus
