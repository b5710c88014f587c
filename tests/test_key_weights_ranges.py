"""How the key weights' steps are cut into the CTAs' ranges (key_weights_ranges.h),
built with the host compiler and compared with counting them one by one."""

import os
import random
import shutil
import subprocess

import numpy as np
import pytest

from causal_gqa_prefill_gb300.build import CSRC

CTAS, KEYS, ROWS = 152, 256, 128

DRIVER = r"""
#include <cstdio>
#include "key_weights_ranges.h"
using namespace gb300_key_weights;
int main() {
  long long heads;
  Shape s;
  while (std::scanf("%d %d %d %d %d %lld", &s.off, &s.nr, &s.steps, &s.T, &s.causal, &heads) == 6) {
    Starts st;
    bool cut;
    const int G = cut_ranges(s, heads, &st, &cut);
    std::printf("%d %d", G, cut ? 1 : 0);
    for (int c = 0; c < G; ++c) std::printf(" %d %d %d", st.unit[c], st.step[c], st.count[c]);
    std::printf("\n");
  }
}
"""


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    at = tmp_path_factory.mktemp("ranges")
    (at / "driver.cpp").write_text(DRIVER)
    exe = str(at / "driver")
    subprocess.run([shutil.which("g++") or "c++", "-std=c++17", "-O1", "-Wall", "-Werror",
                    "-I" + CSRC, str(at / "driver.cpp"), "-o", exe], check=True)

    def run(cases):
        text = "".join("%d %d %d %d %d %d\n" % c for c in cases)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        return [[int(x) for x in line.split()] for line in out.splitlines()]

    return run


def shape(Lq, Lk, g, causal, heads):
    nr = ROWS // g
    return Lk - Lq, nr, -(-Lq // nr), -(-Lk // KEYS), int(causal), heads


def counted(off, nr, steps, T, causal, heads):
    """The same from the definition: every unit's steps, laid end to end."""
    first = np.maximum(np.arange(T, dtype=np.int64) * KEYS - off, 0) // nr if causal else \
        np.zeros(T, dtype=np.int64)
    ends = np.cumsum(steps - first)
    per_head = int(ends[-1])
    W = per_head * heads
    G = min(CTAS, W)
    out, cut = [], 0
    for c in range(G):
        x = c * W // G
        head, rest = divmod(x, per_head)
        t = int(np.searchsorted(ends, rest, side="right"))
        step = int(first[t] + rest - (ends[t] - (steps - first[t])))
        cut |= step != first[t]
        out += [head * T + t, step, (c + 1) * W // G - x]
    return [G, int(cut)] + out


CASES = [
    # Lq, Lk, g, causal, heads
    (300, 300, 4, True, 1),
    (8192, 8192, 4, True, 8),
    (8192, 8192, 7, True, 3),
    (777, 777, 12, True, 2),
    (2048, 8192, 4, True, 8),
    (60, 1300, 12, True, 64),           # fewer positions than a unit's keys
    (131072, 131072, 1, True, 8),
    (131072, 131072, 128, True, 1),     # one position a step
    (3, 700, 128, True, 60),
    (9000, 9001, 3, False, 5),
    (257, 1 << 20, 1, True, 1),
    (300000, 1 << 20, 5, True, 3000),   # 1.4e11 steps (at most 2^30 a CTA are accepted)
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_starts_against_counting(driver, case):
    s = shape(*case)
    assert driver([s]) == [counted(*s)]


def test_random_shapes(driver):
    rng = random.Random(1)
    shapes = []
    for _ in range(400):
        g = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 31, 64, 65, 128])
        Lk = int(2 ** rng.uniform(1, 17))
        Lq = rng.choice([Lk, rng.randint(1, Lk), min(Lk, rng.randint(1, 600))])
        shapes.append(shape(Lq, Lk, g, rng.random() < 0.8, rng.randint(1, 40)))
    for s, got in zip(shapes, driver(shapes)):
        assert got == counted(*s), s
