"""What the axes of qk_norm_rope_axes may be (CPU only)."""
import os

import numpy as np
import pytest
import torch

from conftest import ROOT

LIB = os.path.join(ROOT, "column_scaled_gemm_amd", "libfp8sm.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libfp8sm.so not built")


@pytest.mark.timeout(20)
@pytest.mark.parametrize("mixed", [True, False])
def test_sections_are_numbers_of_pairs(mixed):
    from column_scaled_gemm_amd import fp8sm
    for sections in ([-1, 3], [2, 3, -2], np.array([4, -4])):
        with pytest.raises(ValueError):
            fp8sm.rope_axes(sections, mixed)
    for sections in ([1.5, 2], [2.0], ["2"]):
        with pytest.raises(TypeError):
            fp8sm.rope_axes(sections, mixed)
    assert sorted(fp8sm.rope_axes(np.array([3, 0, 2]), mixed)) == [0, 0, 0, 2, 2]
