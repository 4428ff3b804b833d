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


def test_the_axes_are_host_integers_of_any_kind():
    """Of a numpy array its numbers count, not its memory; a single number names no pair."""
    from column_scaled_gemm_amd import fp8sm
    x, t = torch.zeros(5, 192, dtype=torch.bfloat16), torch.zeros(8, 64)
    pos = torch.zeros(2, 5, dtype=torch.int32)
    for axes in ([0, 1] * 16, (0, 1) * 16, np.array([0, 1] * 16), np.array([0, 1] * 16, dtype=np.uint8),
                 torch.tensor([0, 1] * 16), bytes(32), bytearray(32)):
        with pytest.raises(fp8sm.DeviceTensorError):           # (the tensors are the host's: the next check)
            fp8sm.qk_norm_rope_axes(x, 2, 1, 64, pos, t, axes)
    for axes in (np.zeros(4, dtype=np.int64), np.zeros(16, dtype=np.int16), [0, 256] * 16, [0, -1] * 16):
        with pytest.raises(ValueError):
            fp8sm.qk_norm_rope_axes(x, 2, 1, 64, pos, t, axes)
    for axes in (32, [0.0, 1.0] * 16, None):
        with pytest.raises(TypeError):
            fp8sm.qk_norm_rope_axes(x, 2, 1, 64, pos, t, axes)
