"""The merge of a shared prefix forms addresses from the rows' entries in the workspace.
An attention whose wait ran out leaves entries unwritten: whatever lies there, what the
merge accepts stays inside the workspace.  Checked on the host with the predicate that
the kernel calls (csrc/paged.h)."""
import os
import random
import subprocess

import pytest

from decode_qwen2_block_gb300 import build as gpu_build

PROGRAM = r"""
#include <stdio.h>
#include "paged.h"
int main() {
  int c0, c1, row, nc, rows, G;
  while (scanf("%d %d %d %d %d %d", &c0, &c1, &row, &nc, &rows, &G) == 6)
    printf("%d\n", (int)blk::paged_row_part(c0, c1, row, nc, rows, G));
}
"""


@pytest.fixture(scope="module")
def accepted(tmp_path_factory):
    d = tmp_path_factory.mktemp("merge")
    (d / "t.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", gpu_build.CSRC, "-I",
                    os.path.join(gpu_build.CUDA, "include"), str(d / "t.cpp"), "-o", str(d / "t")],
                   check=True)

    def run(entries):
        text = "\n".join(" ".join(map(str, e)) for e in entries)
        out = subprocess.run([str(d / "t")], input=text, capture_output=True, text=True, check=True)
        return [int(v) for v in out.stdout.split()]
    return run


def test_accepted_entries_stay_inside_the_workspace(accepted):
    rng = random.Random(1)
    edge = [-2 ** 31, -2, -1, 0, 1, 15, 16, 255, 256, 303, 304, 2 ** 30, 2 ** 31 - 1]
    entries = []
    for nc, rows, G in ((304, 16, 6), (304, 32, 16), (152, 256, 1), (152, 256, 16), (7, 16, 1)):
        for _ in range(6000):
            pick = lambda: rng.choice([rng.choice(edge), rng.randrange(-4, nc + 4),  # noqa: E731
                                       rng.randrange(-2 ** 31, 2 ** 31)])
            entries.append((pick(), pick(), pick(), nc, rows, G))
    got = accepted(entries)
    assert len(got) == len(entries) and 0 < sum(got) < len(got)
    for (c0, c1, row, nc, rows, G), ok in zip(entries, got):
        if ok and c0 != -1:
            pieces = c1 - c0 + 1
            assert 1 <= pieces <= nc
            for hh in (0, G - 1):
                first, last = (c0 * 2 + 1) * rows + row + hh, c1 * 2 * rows + row + hh
                assert 0 <= first < nc * 2 * rows and 0 <= last < nc * 2 * rows
                assert row + hh < rows


def test_every_entry_that_the_kernels_write_is_accepted_and_no_part_is_not(accepted):
    entries, want = [], []
    for nc, rows, G in ((304, 16, 6), (304, 32, 16), (152, 256, 6)):
        for c0, c1 in ((0, 0), (0, 1), (3, nc - 1), (nc - 1, nc - 1)):
            for row in (0, G, rows - G):
                entries.append((c0, c1, row, nc, rows, G))
                want.append(1)
        entries += [(-1, 5, 0, nc, rows, G), (-2, 0, 0, nc, rows, G)]
        want += [1, 0]
    assert accepted(entries) == want
