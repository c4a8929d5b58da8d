"""How lora_add is cut up over the device (plain host code), compiled and run here."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "lora_cut.cuh"
using namespace qsm::lora;
// a device of 152 SMs that holds `each` of the CTAs on one
static long long g_each;
static long long clusters(int cs) { return g_each * (cs == 2 ? 76 : cs == 4 ? 37 : 18); }
int main() {
  long long cases = 0, wrong = 0;
  for (g_each = 1; g_each <= 2; ++g_each)
    for (long long T = 1; T <= 40000; T += T < 70 ? 1 : T / 7)
      for (int n : {1, 2, 5, 16, 63, 64, 100, 255, 1000, 1023, 1024, 5000})
        for (int N : {1, 40, 2048, 2050, 8192, 65536}) {
          const bool items = grouped(T, n);
          const long long singles = 152 * g_each, tile = T < 64 ? T : 64;
          const Cut c = cut(items, T, n, N, singles, clusters);
          const long long held = c.cs == 1 ? singles : clusters(c.cs);
          const long long most = T / 64 + (n + 1 < T ? n + 1 : T);  // items, with the largest tile
          const bool even = c.cs == 1 || c.cs == 2 || c.cs == 4 || c.cs == 8;
          ++cases;
          if (!even || c.ctas < 1 || c.parts < 1 || c.lanes < 1 || c.room < 1) ++wrong;
          if ((c.parts > 1 ? c.room * c.parts : c.room) > held) ++wrong;   // what is planned for runs at once
          if (items && (c.lanes < most || c.lanes < c.room || c.ctas != (long long)c.lanes * c.parts * c.cs)) ++wrong;
          if (!items && c.ctas != (T + tile - 1) / tile * c.lanes * c.parts * c.cs) ++wrong;
          if (c.parts > 1 && c.ctas > held * c.cs) ++wrong;                // parts only in one wave
        }
  std::printf("%lld %lld ", cases, wrong);
  // no room: nothing to launch
  std::printf("%lld\n", cut(true, 100, 4, 64, 0, [](int) { return 0ll; }).ctas);
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ missing")
def test_no_more_is_planned_than_the_device_holds(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "quantized_sparse_moe_gb300", "csrc"), str(src), "-o", str(exe)], check=True)
    cases, wrong, none = map(int, subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split())
    assert cases > 5000 and wrong == 0 and none == 0
