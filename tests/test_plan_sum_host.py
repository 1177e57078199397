"""The token plan's sums on the CPU: the prefix sum over a wave's 64 requests,
step by step as the kernel forms it, with the kernel's own cut_sum (compiled
here from csrc/plan_sum.h with signed overflow trapped), against Python's
integers."""
import os
import shutil
import subprocess

import numpy as np
import pytest

import bit_nf4_quantized_07_amd as q

CSRC = os.path.join(os.path.dirname(q.__file__), "csrc")
SRC = """
#include <cstdio>
#include "plan_sum.h"
// stdin: M, what came before, 64 lengths; stdout: the end of each request
int main() {
  int M, before, v[64];
  while (scanf("%d %d", &M, &before) == 2) {
    for (int& x : v) if (scanf("%d", &x) != 1) return 1;
    for (int d = 1; d < 64; d <<= 1) {
      int o[64];
      for (int l = 0; l < 64; ++l) o[l] = l >= d ? qlk::cut_sum(v[l], v[l - d], M) : v[l];
      for (int l = 0; l < 64; ++l) v[l] = o[l];
    }
    for (int l = 0; l < 64; ++l) printf("%d ", qlk::cut_sum(before, v[l], M));
    printf("\\n");
  }
}
"""
TOP = 1 << 30      # the largest M and the largest length after its cut
CASES = [
    (TOP, 0, [TOP, TOP]), (TOP, TOP, [TOP] * 64), (TOP, 5, [TOP - 5, 1, TOP]), (TOP, 0, [TOP]),
    (TOP, 0, [TOP // 2, TOP // 2, 0, 7]), (TOP, 0, [TOP - 1, 1, 1]), (TOP - 1, 3, [TOP - 1] * 3),
    (1, 0, [1, 1]), (7, 7, [0, 7]), (500, 20, list(np.random.default_rng(1).integers(0, 40, 64))),
]


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_prefix_sum_at_the_largest_sizes(tmp_path):
    src, exe = tmp_path / "sum.cpp", tmp_path / "sum"
    src.write_text(SRC)
    subprocess.run(["g++", "-std=c++17", "-O1", "-ftrapv", f"-I{CSRC}", str(src), "-o", str(exe)],
                   check=True)
    rows = [(M, b, [int(x) for x in v] + [0] * (64 - len(v))) for M, b, v in CASES]
    text = "\n".join(" ".join(map(str, (M, b, *v))) for M, b, v in rows) + "\n"
    out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
    got = [[int(x) for x in line.split()] for line in out.splitlines()]
    for (M, b, v), g in zip(rows, got, strict=True):
        assert g == [min(M, b + sum(v[:l + 1])) for l in range(64)], (M, b, v)
