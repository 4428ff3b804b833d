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


ORDER = r"""
#define __host__
#define __device__
#include "packed_rows.h"
#include <cstdio>
int main(int argc, char** argv) {
  long long T;
  int prompts, heads, D;
  while (std::scanf("%lld %d %d %d", &T, &prompts, &heads, &D) == 4)
    std::printf("%d\n", (int)fp8sm::heads_side_by_side(T, prompts, heads, D));
  return 0;
}
"""


def run(tmp_path, program, given=""):
    src, exe = tmp_path / "rows.cpp", str(tmp_path / "rows")
    src.write_text(program)
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "column_scaled_gemm_amd", "csrc"), str(src), "-o", exe],
                   check=True)
    return subprocess.run([exe], check=True, capture_output=True, text=True, input=given).stdout.split()


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_the_order_of_the_heads_counts_their_keys(tmp_path):
    """The heads follow each other only where their keys and values of a prompt outgrow the
    last-level cache: that takes tokens, not heads alone."""
    cases = [(500, 1, 112, 128, 1), (8100, 1, 128, 128, 0), (8100, 27, 128, 128, 1), (2000, 1, 128, 128, 1),
             (4160, 1, 224, 128, 0), (8320, 2, 192, 128, 0), (1000, 1, 128, 64, 1), (8320, 1, 56, 128, 1),
             (8320, 1, 112, 128, 0), (65536, 1, 8, 128, 1), (8388608, 1, 64, 128, 1), (1, 1, 1024, 128, 1),
             (1048576, 1, 1024, 128, 0), (3, 1048576, 1024, 128, 1)]
    got = run(tmp_path, ORDER, "".join(" ".join(map(str, c[:4])) + "\n" for c in cases))
    assert [int(x) for x in got] == [c[4] for c in cases]


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_a_workgroup_reads_queries_of_its_own_rows(tmp_path):
    """With o in q's place another workgroup's rows are being written while this one runs:
    lanes behind the prompt's last row read a row of their own tile."""
    seen, bad = map(int, run(tmp_path, PROGRAM))
    assert seen > 100000 and bad == 0
