"""Pins of the int8 oracle (CPU only)."""
import numpy as np
import pytest

from oracle import bf16, fp16, int8 as oi

F32 = np.float32


@pytest.mark.parametrize("e", [-20, -3, 0, 5, 40])
def test_rows_of_integers_times_a_power_of_two_come_back(e):
    k = np.arange(-127, 128, dtype=F32)
    q, s = oi.quant((k * F32(2.0 ** e))[None])
    assert np.array_equal(q[0], k.astype(np.int8)) and s[0] == F32(2.0 ** e)


def test_ties_go_to_even_and_signs_mirror():
    y = np.array([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5]], dtype=F32)
    q, s = oi.quant(y)
    assert q[0].tolist() == [127, 0, 2, 2, 0, -2, -2, 126] and s[0] == 1
    assert np.array_equal(oi.quant(-y)[0], -q)


def test_floor_and_values_that_are_not_finite():
    q, s = oi.quant(np.array([[0.0, 0.0], [1e-12, -1e-12]], dtype=F32))
    assert not q[0].any() and s[0] == F32(1e-10) / F32(127) and q[1].tolist() == [1, -1]
    q, s = oi.quant(np.array([[np.inf, -np.inf, np.nan, 127.0, -1.0], [np.inf] * 2 + [np.nan] * 3], dtype=F32))
    assert q[0].tolist() == [127, -127, 0, 127, -1] and s[0] == 1
    assert q[1].tolist() == [127, 127, 0, 0, 0] and s[1] == F32(1e-10) / F32(127)


def test_codes_are_within_half_a_step_of_the_value():
    r = np.random.Generator(np.random.PCG64(3))
    y = r.standard_normal((50, 333)).astype(F32) * F32(7)
    q, s = oi.quant(y)
    # two fp32 roundings of the multiplier and the product move a code's value by at
    # most 127 * 2^-23 of a step
    assert np.all(np.abs(y / s[:, None].astype(np.float64) - q) <= 0.5 + 127 * 2.0 ** -22)
    assert np.array_equal(np.abs(q).max(1), np.full(50, 127))


def test_products_are_the_sums_of_python_integers():
    r = np.random.Generator(np.random.PCG64(4))
    a = r.integers(-128, 128, (3, 40)).astype(np.int8)
    b = r.integers(-128, 128, (5, 40)).astype(np.int8)
    want = [[sum(int(x) * int(y) for x, y in zip(ra, rb)) for rb in b] for ra in a]
    assert oi.product(a, b).tolist() == want
    top = np.full((1, 65536), -128, dtype=np.int8)
    assert oi.product(top, top)[0, 0] == 2 ** 30


def test_scaled_output_of_exact_cases():
    a, b = np.array([[2, 3]], np.int8), np.array([[5, -7], [1, 1]], np.int8)
    bits = oi.scaled_mm(a, b, [0.5], [2.0, 4.0], bias=[1.0, -2.0])
    assert bf16.bits_to_f64(bits).tolist() == [[-10.0, 8.0]]
    bits = oi.scaled_mm(a, b, 0.5, 2.0, out="fp16")
    assert fp16.bits_to_f64(bits).tolist() == [[-11.0, 5.0]]
