"""The paged attention's work split as the kernels have it (csrc/attn_paged_split.h, compiled for the host)
against the plan of test_generation_schedule.py: shares and owners of every place, what lies at a place, and
the parts that each CTA leaves."""
import os
import random
import shutil
import subprocess

import pytest

from io_aware_attention_attn_gb300 import build
from test_generation_schedule import join, plan, shares, walk

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "attn_paged_split.h"
using namespace attn;
// per case: requests, K/V heads, row groups, CTAs, cost, then the requests' tiles
int main() {
  int B, H, R, ctas, cost;
  while (std::scanf("%d %d %d %d %d", &B, &H, &R, &ctas, &cost) == 5) {
    std::vector<int> tiles(B), first(B + 1, 0);
    for (int s = 0; s < B; ++s) {
      std::scanf("%d", &tiles[s]);
      first[s + 1] = first[s] + (tiles[s] + cost) * H * R;
    }
    const int total = first[B], G = ctas < total ? ctas : total;
    const Shares sh(total, G);
    std::printf("G %d\n", G);
    for (int i = 0; i <= G; ++i) std::printf("%d ", sh.start(i));
    std::printf("\n");
    for (int p = 0; p < total; ++p) std::printf("%d ", sh.owner(p));
    std::printf("\n");
    for (int s = 0, p = 0; p < total; ++p) {
      while (p >= first[s + 1]) ++s;
      const UnitAt u = unit_at(p - first[s], tiles[s] + cost, R);
      std::printf("%d:%d ", (s * H + u.h) * R + u.rg, u.t);
    }
    std::printf("\n");
    for (int i = 0; i < G; ++i) {  // the parts' kernel, one CTA after another
      int s = 0, place = sh.start(i), left = sh.start(i + 1) - place;
      while (place >= first[s + 1]) ++s;
      UnitAt u = unit_at(place - first[s], tiles[s] + cost, R);
      int unit = (s * H + u.h) * R + u.rg, t = u.t;
      const int unit0 = place - t;
      if (t >= tiles[s]) {
        left -= unit0 + tiles[s] + cost - place;
        if (left <= 0) { std::printf("\n"); continue; }
        ++unit, t = 0;
      }
      while (left > 0) {
        const int n = tiles[unit / (H * R)], end = n < t + left ? n : t + left;
        std::printf("%d:%d:%d ", unit, t, end);
        left -= places_done(t, end, n, cost);
        ++unit, t = 0;
      }
      std::printf("\n");
    }
    for (int s = 0; s < B; ++s)  // and what the join takes for the first part of a unit
      for (int k = 0; k < H * R; ++k) {
        const int unit0 = first[s] + k * (tiles[s] + cost), i0 = sh.owner(unit0);
        std::printf("%d:%d:%d ", i0, sh.owner(unit0 + tiles[s] - 1), second_part(sh.start(i0), unit0, cost));
      }
    std::printf("\n");
  }
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    cxx = os.environ.get("CXX", "g++")
    if shutil.which(cxx) is None:
        pytest.skip("needs a host compiler")
    at = tmp_path_factory.mktemp("split")
    (at / "split.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-Wno-unused-result", "-I", build.CSRC,
                    str(at / "split.cpp"), "-o", str(at / "split")], check=True)
    return str(at / "split")


def cases():
    r = random.Random(1)
    for _ in range(150):
        B, H, R = r.randint(1, 30), r.choice([1, 2, 5, 8]), r.choice([1, 1, 2, 3])
        top = r.choice([1, 3, 20, 120])
        yield ([max(1, r.randint(0, top)) for _ in range(B)], H, R, r.choice([1, 2, 7, 152, 304, 456, 608]),
               r.choice([0, 1, 2]))


def test_split_of_the_kernels_is_the_plan(program):
    todo = list(cases())
    text = "".join(f"{len(t)} {H} {R} {ctas} {cost} {' '.join(map(str, t))}\n" for t, H, R, ctas, cost in todo)
    out = iter(subprocess.run([program], input=text, capture_output=True, text=True, check=True).stdout.split("\n"))

    def line():
        return [tuple(map(int, w.split(":"))) for w in next(out).split()]

    for tiles, H, R, ctas, cost in todo:
        units, total, G = plan(tiles, H * R, ctas, cost)
        start, owner = shares(total, G)
        assert next(out) == f"G {G}"
        assert [x for x, in line()] == [start(i) for i in range(G + 1)]
        assert [x for x, in line()] == [owner(p) for p in range(total)]
        assert line() == [(u, t) for u, (_, n) in enumerate(units) for t in range(n + cost)]
        for cta in range(G):
            assert line() == walk(units, total, G, cost, cta)
        for u, (i0, i1, second) in enumerate(line()):
            j = join(units, total, G, cost, u, True)
            assert (j is None) == (i0 == i1)
            if j is not None:
                assert j == (u, [(i, second if i == i0 else 0) for i in range(i0, i1 + 1)])
    assert next(out) == ""
