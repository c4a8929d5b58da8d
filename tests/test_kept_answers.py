"""The table of kept occupancy answers (plain host code), compiled and run here."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include "kept_answers.cuh"
using qsm::mx4::KeptAnswers;
static KeptAnswers t;
static char kernels[4];
int main() {
  // what several projections (K = 256 .. 4096) with 1 to 32 rows ask for, over and
  // over: each is asked for once
  int misses = 0, wrong = 0, asked = 0;
  for (int round = 0; round < 3; ++round)
    for (int k = 1; k <= 16; ++k)
      for (int rows = 1; rows <= 32; ++rows)
        for (int cs = 1; cs <= 8; cs *= 2) {
          const int segs = (k + cs - 1) / cs, smem = 7 * 17408 + segs * (rows * 768 + 1024) + (cs > 1 ? rows * 1024 : 0);
          int n = -1;
          ++asked;
          if (!t.find(0, &kernels[0], cs, smem, &n)) {
            ++misses;
            t.put(0, &kernels[0], cs, smem, cs * 1000000 + smem);
          } else if (n != cs * 1000000 + smem) {
            ++wrong;
          }
        }
  std::printf("%d %d %d ", asked, misses, wrong);
  // device and kernel belong to the question
  int n = 0;
  t.put(1, &kernels[1], 2, 5, 7);
  std::printf("%d%d%d%d ", t.find(1, &kernels[1], 2, 5, &n), t.find(0, &kernels[1], 2, 5, &n),
              t.find(1, &kernels[2], 2, 5, &n), t.find(1, &kernels[1], 4, 5, &n));
  // more than fit: answers get lost, never mixed up
  static KeptAnswers full;
  const int many = 3 * KeptAnswers::kSlots;
  int lost = 0;
  for (int i = 0; i < many; ++i) full.put(0, &kernels[3], 1, i, i + 1);
  for (int i = 0; i < many; ++i) {
    if (!full.find(0, &kernels[3], 1, i, &n)) ++lost;
    else if (n != i + 1) ++wrong;
  }
  std::printf("%d %d\n", wrong, lost == many - (int)KeptAnswers::kSlots);
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ missing")
def test_every_geometry_is_asked_for_once(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "quantized_sparse_moe_gb300", "csrc"), str(src), "-o", str(exe)], check=True)
    asked, misses, wrong, parts, wrong_full, lost = subprocess.run(
        [str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert (int(asked), int(wrong), parts, int(wrong_full), int(lost)) == (6144, 0, "1000", 0, 1)
    assert int(misses) <= 2048                     # the first round's
