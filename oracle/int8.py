"""Per-token int8 quant and the scaled int8 product.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Definitions (include/fp8sm.h): with a' = max(max|y|, 1e-10) over the finite y of a
row, scale = RN32(a' / 127) and code = the integer nearest RN32(y * RN32(127 / a')),
ties to even; an infinity +-127, a NaN 0.  The product is exact in integers, then
RN32(RN32(RN32(acc) sa) sb) + bias in fp32, rounded once to the output type.

Pins (tests/test_oracle_int8.py): closed forms of rows whose largest value is 127
times a power of two, codes' ties, sign symmetry, scaling by powers of two, products
against sums in Python integers.
"""
import numpy as np

from . import bf16, fp16

F32 = np.float32


def quant(y32):
    """[..., K] float32 -> (codes int8 [..., K], scales float32 [...])."""
    y = np.asarray(y32, dtype=F32)
    finite = np.isfinite(y)
    top = np.where(finite, np.abs(y), F32(0)).max(-1)
    a = np.maximum(top, F32(1e-10)).astype(F32)
    mult = (F32(127) / a).astype(F32)
    with np.errstate(invalid="ignore", over="ignore"):
        v = np.rint((y * mult[..., None]).astype(F32))
    v = np.where(np.isnan(y), F32(0), np.clip(v, F32(-127), F32(127)))
    return np.nan_to_num(v).astype(np.int8), (a / F32(127)).astype(F32)


def product(a, b):
    """[M, K] x [N, K] int8 -> exact sums, int64."""
    # float64 holds every partial sum (below 2^31) exactly
    return np.rint(np.asarray(a, np.float64) @ np.asarray(b, np.float64).T).astype(np.int64)


def scaled_mm(a, b, sa, sb, bias=None, out="bf16"):
    """16-bit patterns [M, N] of the output; sa, sb: vectors or scalars."""
    acc = product(a, b).astype(F32)
    sa, sb = (np.asarray(s, dtype=F32).reshape(-1) for s in (sa, sb))
    with np.errstate(over="ignore", invalid="ignore"):
        y = ((acc * sa[:, None]).astype(F32) * sb[None, :]).astype(F32)
        if bias is not None:
            y = (y + np.asarray(bias, dtype=F32)[None, :]).astype(F32)
    return bf16.to_bf16_bits(y) if out == "bf16" else fp16.to_fp16_bits(y)
