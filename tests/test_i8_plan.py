"""The choice of gdn_linear_i8's kernels (csrc/gdn_linear_i8_plan.h, plain host
code) over the sizes it accepts, and that the shapes of the tests reach every
kernel that it can choose."""
import ast
import os
import random
import subprocess

import pytest

import i8_shapes
from linear_attention_recurrence_04_b200 import build as gdn_build

SMS = 148
VEC, SPLIT, PAIR = range(3)
MAIN = r"""
#include <cstdio>
#include "gdn_linear_i8_plan.h"
int main() {
    long long M, N, K, sms;
    while (std::scanf("%lld %lld %lld %lld", &M, &N, &K, &sms) == 4) {
        const gdn::PlanI8 p = gdn::plan_i8(M, N, K, sms);
        std::printf("%d %d %d %d\n", static_cast<int>(p.form), p.tile, p.splits, gdn::vec_warps(K));
    }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "main.cpp").write_text(MAIN)
    exe = str(d / "plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", gdn_build.CSRC, "-o", exe,
                    str(d / "main.cpp")], check=True)

    def ask(shapes, sms=SMS):
        text = "".join(f"{M} {N} {K} {sms}\n" for M, N, K in shapes)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return ask


def test_shapes_reach_their_kernels(plan):
    got = plan([s[:3] for s in i8_shapes.SPLIT])
    for s, p in zip(i8_shapes.SPLIT, got):
        assert p[:3] == (SPLIT, s[3], s[4]), (s, p)
    for s, p in zip(i8_shapes.VEC, plan([s[:3] for s in i8_shapes.VEC])):
        assert p[0] == VEC and p[3] == s[4], (s, p)
    for s, p in zip(i8_shapes.PAIR, plan([s[:3] for s in i8_shapes.PAIR])):
        assert p[:2] == (PAIR, s[3]), (s, p)
    # what the lists are for
    for tile in (16, 32, 64, 128):
        for splits in (1, 2, 4, 8):
            own = [s for s in i8_shapes.SPLIT if s[3:] == (tile, splits)]
            assert {min(s[1] % 4, 2) if s[1] % 2 == 0 else 1 for s in own} == {0, 1, 2}, (tile, splits)
            assert any(s[2] % 32 == 16 and s[0] % tile for s in own)
            assert splits == 1 or any(-(-s[2] // 256) % splits for s in own)
    for tile in (128, 256):
        assert {s[1] % 16 for s in i8_shapes.PAIR if s[3] == tile} >= {0, 8, 12, 10, 11}


def reaches(p, M):
    """What tells one kernel from another: its template arguments and the
    number of CTAs."""
    tokens = 1 if M == 1 else 2 if M == 2 else 4 if M <= 4 else 8
    return ("vec", tokens, p[3]) if p[0] == VEC else ("split", *p[1:3]) if p[0] == SPLIT else ("pair", p[1])


def test_nothing_is_reached_but_what_is_tested(plan):
    """Random sizes over the accepted range choose no kernel that the lists do
    not, and choose each of them: none is there for nothing."""
    lists = i8_shapes.SPLIT + i8_shapes.VEC + i8_shapes.PAIR
    tested = {reaches(p, s[0]) for s, p in zip(lists, plan([s[:3] for s in lists]))}
    rng = random.Random(0)

    def log(lo, hi):
        return round(lo * (hi / lo) ** rng.random())
    shapes = [(log(1, 65535 * 128), log(1, 200000), 16 * log(1, 8191)) for _ in range(150000)]
    shapes += [(log(1, 4000), log(1, 4000), 16 * log(1, 700)) for _ in range(150000)]
    got = plan(shapes)
    assert {reaches(p, s[0]) for s, p in zip(shapes, got)} == tested
    # a cluster's CTAs all have a k-step of their own, and the grids fit 32 bits
    for (M, N, K), (form, tile, splits, warps) in zip(shapes, got):
        if form == SPLIT:
            assert 1 <= splits <= min(8, -(-K // 256))
            assert -(-N // 128) * -(-M // tile) * splits < 2 ** 31
        elif form == VEC:
            mt = 1 if M == 1 else 2 if M == 2 else 4 if M <= 4 else 8
            rows = 4 // warps * (4 if mt == 4 or mt == 8 and warps == 4 else 2)
            assert -(-N // rows) * -(-M // mt) < 2 ** 31
        else:
            assert M > 128 and -(-N // tile) * -(-M // 256) < 2 ** 30


def test_other_numbers_of_sms(plan):
    """On fewer SMs the choice is still one of the forms."""
    shapes = [s[:3] for s in i8_shapes.SPLIT + i8_shapes.PAIR]
    for sms in (2, 20, 142):
        for (M, N, K), (form, tile, splits, _) in zip(shapes, plan(shapes, sms)):
            assert form in (VEC, SPLIT, PAIR)
            assert form != SPLIT or (tile in (16, 32, 64, 128) and splits in (1, 2, 4, 8))


def test_smoke_reaches_every_form(plan):
    """The shapes that __graft_entry__.smoke() runs."""
    with open(os.path.join(gdn_build.ROOT, "__graft_entry__.py")) as f:
        tree = ast.parse(f.read())
    lists = [n.value for n in ast.walk(tree) if isinstance(n, ast.Assign)
             and any(getattr(t, "id", "") == "I8_SHAPES" for t in n.targets)]
    shapes = ast.literal_eval(lists[0])
    got = plan(shapes)
    assert {p[0] for p in got} == {VEC, SPLIT, PAIR}
    assert {p[2] > 1 for p in got if p[0] == SPLIT} == {True}
