"""The kernel that the int8 product picks for a size (CPU only)."""
import os
import random

import pytest

from conftest import ROOT

LIB = os.path.join(ROOT, "column_scaled_gemm_amd", "libfp8sm.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libfp8sm.so not built")


def workgroups(name, M, N):
    """(workgroups of a batch in a grid's first dimension, threads of each)."""
    bm, bn = map(int, name.split()[-1 if name.startswith("few") else 0].split("x"))
    n = -(-N // bn) if name.startswith("few") else -(-M // bm) * -(-N // bn)
    return n, 256 if name == "64x32" else 512


def corners():
    top = 1 << 30                     # of a dimension; outputs: 2^37
    for n in (8, 16, 32, 64, 72, 120, 128):
        yield from ((m, n) for m in (top, top - 1, top - 127, top - 128, top // 2 + 1))
    for m in (1, 16, 17, 33, 64, 65, 127, 128):
        yield from ((m, n) for n in (top, top - 8, top - 120, top - 128, top // 2 + 8, 1 << 26, (1 << 26) + 8))
    r = random.Random(1)
    for _ in range(2000):
        m = min(top, int(2 ** r.uniform(0, 30.1)))
        yield m, max(8, min(top, int(2 ** r.uniform(3, 30.1)), (1 << 37) // m) // 8 * 8)


def test_a_launch_holds_less_than_2_to_32_threads():
    from column_scaled_gemm_amd import fp8sm
    for M, N in corners():
        for batches in (1, 2, 64, 65535):
            name = fp8sm.int8_kernel(batches, M, N)
            n, threads = workgroups(name, M, N)
            assert n * threads < 1 << 32, (batches, M, N, name)
