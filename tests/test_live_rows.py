"""The live-row counts of the batched calls lie one behind the other in memory (CPU only)."""
import pytest
import torch

from column_scaled_gemm_amd import fp8sm


class OnDevice:
    """A tensor of the host that says that it is a device's."""
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_counts_with_a_stride_are_refused():
    """The kernels read B consecutive counts: of every second one they would take others,
    of one that is expanded they would read past its memory."""
    whole = torch.arange(8, dtype=torch.int32)
    good = OnDevice(whole)
    assert fp8sm._rows_arg(good, 8) is good
    one = OnDevice(whole[3:4].expand(1))
    assert fp8sm._rows_arg(one, 1) is one
    for t, B in ((whole[::2], 4), (whole[:1].expand(8), 8)):
        with pytest.raises(ValueError):
            fp8sm._rows_arg(OnDevice(t), B)
