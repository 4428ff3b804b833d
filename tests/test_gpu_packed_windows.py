"""Packed attention through a window: what a row does not see, behind it or before its
window, does not reach it, whatever it holds."""
import numpy as np
import pytest
import torch

from column_scaled_gemm_amd import fp8sm
from kv_util import DT, rng

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 100, 190])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_a_bad_value_reaches_the_rows_whose_window_holds_it(window, D, dtype):
    print("[case] window", window, D, dtype, flush=True)
    r = rng(window + D)
    cu, Hq, H = [0, 130, 530, 607], 4, 2
    T, end = cu[-1], cu[2]
    q, k, v = (torch.from_numpy(r.standard_normal((T, h, D)).astype(np.float32)).cuda().to(DT[dtype]) for h in (Hq, H, H))
    starts = torch.tensor(cu, dtype=torch.int32, device="cuda")

    def call(k, v):
        return fp8sm.attention_packed(q, k, v, starts, window=window, return_lse=True)

    clean, clean_lse = call(k, v)
    assert torch.isfinite(clean).all() and torch.isfinite(clean_lse).all()
    for at in (130, 193, 280, 511, 529):          # of the second prompt
        rows = slice(at, min(at + window, end))
        for bad in (float("nan"), float("inf"), -float("inf")):
            v2 = v.clone()
            v2[at, 1, 5] = bad                    # heads 2 and 3, channel 5
            out, lse = call(k, v2)
            hit = torch.zeros_like(out, dtype=torch.bool)
            hit[rows, 2:, 5] = True
            assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse, clean_lse)
            assert not torch.isfinite(out[hit]).any()
            k2 = k.clone()
            k2[at, 0, 3] = bad                    # heads 0 and 1
            out, lse = call(k2, v)
            hit = torch.zeros_like(lse, dtype=torch.bool)
            hit[rows, :2] = True
            assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])
            if bad != bad:
                assert torch.isnan(out[hit]).all()
