"""Cache and attention calls at the edges of what their documentation allows, as
far as the host decides them (no GPU needed)."""
import os

import pytest

from conftest import ROOT

LIB = os.path.join(ROOT, "column_scaled_gemm_amd", "libfp8sm.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libfp8sm.so not built")


@pytest.mark.parametrize("B,T,Hq,H,D,max_q,max_kv", [
    (512, 512, 64, 8, 128, 1, 131072), (1024, 1024, 64, 8, 128, 1, 131072), (1024, 1024, 64, 8, 128, 1, 1 << 20),
    (256, 2048, 64, 8, 128, 8, 1 << 30), (4096, 4096, 128, 8, 64, 1, 1 << 20), (64, 1 << 20, 64, 8, 128, 1 << 14, 1 << 20),
    (1 << 16, 1 << 20, 8, 8, 128, 4096, 1 << 30), (1, 1, 1024, 1024, 128, 1, 1 << 30), (1, 1 << 20, 1024, 8, 128, 33, 1 << 30)])
def test_workspace_is_bounded(B, T, Hq, H, D, max_q, max_kv):
    from column_scaled_gemm_amd import fp8sm
    for window in (0, 4096, (1 << 31) - 1):
        assert fp8sm.attention_cache_workspace(T, B, Hq, H, D, max_q, max_kv, window) < 512 << 20


def test_workspace_of_few_rows_is_that_of_their_splits():
    from column_scaled_gemm_amd import fp8sm
    row = (128 + 2) * 4
    assert fp8sm.attention_cache_workspace(8, 2, 64, 8, 128, 4, 131072) == 32 * 8 * 64 * row
    assert fp8sm.attention_cache_workspace(64, 64, 32, 8, 128, 1, 16384) == 8 * 64 * 32 * row


@pytest.mark.parametrize("window,means", [(1 << 31, 0), ((1 << 32) + 5, 0), (1 << 62, 0), (1 << 64, 0), ((1 << 31) - 1, 0),
                                          (100, 100)])
def test_windows_beyond_32_bits_bound_nothing(window, means):
    """ctypes would cut them to their lowest bits, 5 tokens for 2^32 + 5."""
    from column_scaled_gemm_amd import fp8sm
    sizes = (8, 2, 64, 8, 128, 4, 131072)
    assert fp8sm.attention_cache_workspace(*sizes, window) == fp8sm.attention_cache_workspace(*sizes, means)


def test_negative_windows_are_refused_whatever_their_size():
    from column_scaled_gemm_amd import fp8sm
    assert [fp8sm._window(w) for w in (-1, -(1 << 31), -(1 << 32), -(1 << 40) + 3)] == [-1] * 4
    assert fp8sm.attention_cache_workspace(8, 2, 64, 8, 128, 4, 131072, -(1 << 32)) == 0


@pytest.mark.parametrize("kw", [dict(T=0), dict(B=0), dict(T=0, B=0)])
def test_an_empty_batch_has_no_longest_sequence(kw):
    from test_abi_kv import _attn, _codes
    lib, E = _codes()
    assert _attn(lib, mq=0, mkv=0, **kw) == E["OK"]
    assert _attn(lib, mq=-1, **kw) == _attn(lib, mkv=-1, **kw) == E["ERR_SHAPE"]
    assert _attn(lib, mq=0) == E["ERR_SHAPE"]


def test_an_output_that_is_not_wanted_is_refused():
    import torch
    from column_scaled_gemm_amd import fp8sm
    c = fp8sm.kv_cache_empty(3, 2, 64, 16, device="cpu")
    i32 = dict(dtype=torch.int32)
    rows = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    args = (c, torch.zeros(3, **i32), torch.zeros(2, **i32), torch.zeros(2, 4, **i32), 5)
    for kw in (dict(k=rows, keys=False), dict(v=rows, values=False)):
        with pytest.raises(ValueError):
            fp8sm.kv_cache_read(*args, **kw)
    with pytest.raises(fp8sm.DeviceTensorError):
        fp8sm.kv_cache_read(*args, keys=False)
