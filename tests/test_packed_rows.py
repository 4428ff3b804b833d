"""The rows that a workgroup of the packed attention reads and writes, from the kernel's
own header in a host program (CPU only)."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#define __host__
#define __device__
#include "packed_rows.h"
int main() {
  long bad = 0, seen = 0;
  for (int G : {1, 2, 3, 5, 7, 8, 40})
    for (int n : {1, 2, 16, 25, 127, 128, 129, 300, 1000})
      for (int hk : {0, 3})
        for (int r0 = 0; r0 < n * G; r0 += 128)
          for (int i = 0; i < 128; ++i) {
            const fp8sm::PackedRow p = fp8sm::packed_row(r0, i, n * G, hk, G);
            const int row = p.tok * G + p.head - hk * G;
            ++seen;
            if (p.head < hk * G || p.head >= (hk + 1) * G || p.ok != (r0 + i < n * G)) ++bad;
            if (p.ok ? row != r0 + i : row < r0 || row >= r0 + 128 || row >= n * G) ++bad;
          }
  std::printf("%ld %ld\n", seen, bad);
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_a_workgroup_reads_queries_of_its_own_rows(tmp_path):
    """With o in q's place another workgroup's rows are being written while this one runs:
    lanes behind the prompt's last row read a row of their own tile."""
    src, exe = tmp_path / "rows.cpp", str(tmp_path / "rows")
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "column_scaled_gemm_amd", "csrc"), str(src), "-o", exe],
                   check=True)
    seen, bad = map(int, subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split())
    assert seen > 100000 and bad == 0
