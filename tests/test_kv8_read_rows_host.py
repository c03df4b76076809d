"""Rows that a read of an 8-bit cache would write over each other are refused.  Checked on
the host with the predicate that the library calls (csrc/kv8.h), against all pairs of
rows."""
import itertools
import os
import random
import subprocess

import pytest

from decode_qwen2_block_gb300 import build as gpu_build

PROGRAM = r"""
#include <stdio.h>
#include "kv8.h"
int main() {
  long long n, H, rs, hs, D, apart;
  while (scanf("%lld %lld %lld %lld %lld %lld", &n, &H, &rs, &hs, &D, &apart) == 6)
    printf("%d\n", (int)blk::kv8_rows_meet(n, H, rs, hs, D, apart));
}
"""


@pytest.fixture(scope="module")
def meet(tmp_path_factory):
    d = tmp_path_factory.mktemp("rows")
    (d / "t.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", gpu_build.CSRC, "-I",
                    os.path.join(gpu_build.CUDA, "include"), str(d / "t.cpp"), "-o", str(d / "t")],
                   check=True)

    def run(calls):
        text = "\n".join(" ".join(map(str, c)) for c in calls)
        out = subprocess.run([str(d / "t")], input=text, capture_output=True, text=True, check=True)
        return [v == "1" for v in out.stdout.split()]
    return run


def by_pairs(n, H, rs, hs, D, apart):
    at = [r * rs + h * hs for r in range(n) for h in range(H)]
    own = any(abs(a - b) < D for a, b in itertools.combinations(at, 2))
    return own or any(abs(apart + b - a) < D for a in at for b in at)


def nested(n, H, rs, hs, D):
    return n == 1 or H == 1 or rs >= (H - 1) * hs + D or hs >= (n - 1) * rs + D


def test_all_pairs_of_rows(meet):
    rng = random.Random(4)
    D, calls = 4, []
    for _ in range(30000):
        n, H = rng.randint(1, 5), rng.randint(1, 4)
        a, b = rng.randint(0, 14), rng.randint(0, 60)
        rs, hs = (a, b) if rng.random() < 0.5 else (b, a)
        if rng.random() < 0.6:              # tight, or with room for another row
            tight, room = rng.choice((D, 2 * D, D + 1)), rng.choice((0, 1, D, 4 * D))
            rs, hs = ((H * tight + room, tight) if rng.random() < 0.5 else (tight, n * tight + room))
        apart = rng.choice((0, rng.randint(-90, 90), H * D, -n * D, D, n * H * D))
        calls.append((n, H, rs, hs, D, apart))
    got = meet(calls)
    assert len(got) == len(calls)
    for c, g in zip(calls, got):
        want = by_pairs(*c)
        if nested(*c[:5]):
            assert g == want, c
        else:
            assert g, c                     # rows through each other: refused, whether they meet or not
    assert 5000 < sum(got) < 25000


def test_layouts_that_are_served(meet):
    """K and V of a packed projection, of one buffer, of contiguous caches, behind one another."""
    for n, H, D in ((1, 1, 64), (1, 8, 64), (7, 1, 128), (1 << 20, 2, 128), (1031, 4, 128)):
        C = n + 5
        ok = [(n, H, H * D, D, D, n * H * D), (n, H, 2 * H * D, D, D, H * D), (n, H, 2 * H * D, 2 * D, D, D),
              (n, H, 20 * H * D, D, D, -H * D), (n, H, D, C * D, D, H * C * D), (n, H, 2 * D, 2 * C * D, D, -D),
              (n, H, D, 2 * C * D, D, C * D)]
        assert not any(meet(ok)), (n, H, D)
        bad = [(n, H, H * D, D, D, 0), (n, H, H * D, D, D, 8), (n, H, D, C * D, D, -D + 8),
               (n, H, H * D, D, D, (n - 1) * H * D + 8), (n, H, D, C * D, D, (H - 1) * C * D)]
        assert all(meet(bad)), (n, H, D)
