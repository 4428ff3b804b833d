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


# (batches, rows, columns) that reach each kernel, its ring's slots (0: no ring)
SIZES = {"few 16x16": ((1, 13, 4088), (5, 16, 264)), "few 16x32": ((1, 9, 8200), (1, 16, 9000)),
         "few 32x16": ((1, 31, 2056), (4, 20, 520)), "64x32": ((1, 100, 4000), (1, 492, 1000)),
         "64x64": ((1, 48, 9000), (3, 200, 1000)), "64x128": ((1, 140, 9000), (1, 190, 9000)),
         "128x64": ((1, 300, 5376), (1, 100, 14336)), "128x128 alone": ((1, 600, 4104), (2, 90, 8200)),
         "128x128": ((1, 2560, 6656), (2, 1700, 5000)), "256x256": ((1, 3406, 7544), (3, 700, 5000))}
SLOTS = {"64x32": 6, "64x64": 4, "64x128": 4, "128x64": 4, "128x128 alone": 4, "128x128": 2, "256x256": 2}


def lengths(name):
    """K at which a kernel's walk has one step, as many as its ring, more, and tails."""
    if name not in SLOTS:                       # eight wavefronts, 256 of K a step
        return 16, 2048, 3 * 2048, 3 * 2048 + 16, 2 * 2048 + 240
    ring = 128 * SLOTS[name]
    return 16, ring, ring + 128, ring + 5 * 128, ring + 5 * 128 + 16, ring + 4 * 128 + 112


@pytest.mark.parametrize("name", SIZES)
def test_the_sizes_that_are_tested_reach_the_kernel_they_name(name):
    """tests/test_gpu_int8_kernels.py runs these."""
    from column_scaled_gemm_amd import fp8sm
    for size in SIZES[name]:
        assert fp8sm.int8_kernel(*size) == name, size
    # the loop that copies, reads and multiplies at once runs from two steps more than slots on
    assert name not in SLOTS or sum(-(-K // 128) >= SLOTS[name] + 2 for K in lengths(name)) >= 3


def test_panels_of_16_columns_count_the_batch():
    """They serve calls whose panels are a CU's one workgroup at most: a batch has its
    panels side by side in the same launch (32 experts of 16 rows x 7168 columns: 14336)."""
    from column_scaled_gemm_amd import fp8sm
    for M, panel in ((1, "few 16x16"), (16, "few 16x16"), (17, "few 32x16"), (32, "few 32x16")):
        for batches, N in ((1, 4096), (2, 2048), (32, 128), (256, 16), (256, 8), (5, 816)):
            assert fp8sm.int8_kernel(batches, M, N) == panel, (batches, M, N)
        for batches, N in ((1, 4104), (2, 2056), (32, 136), (32, 7168), (257, 8), (65535, 8), (8, 4096)):
            assert fp8sm.int8_kernel(batches, M, N) != panel, (batches, M, N)
