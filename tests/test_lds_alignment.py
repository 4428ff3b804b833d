"""The alignment of shared memory that kernels read 16 bytes at a time (CPU only)."""
import os
import re

from column_scaled_gemm_amd import build


def test_the_rotations_cosines_and_sines_are_aligned_for_16_byte_reads():
    """qk_norm_rope_axes gathers a token's cosines and sines into shared memory and reads
    four at a time: their declaration has to promise that (a compiler that aligns large
    arrays by itself, as the present one does, need not)."""
    text = open(os.path.join(build.CSRC, "kv_cache.hip")).read()
    assert "const float4*>(row" in text and "row = AXES ? turns" in text
    declared = re.findall(r"__shared__ ([^;]*)\bturns\[", text)
    assert len(declared) == 1 and "aligned(16)" in declared[0], declared
