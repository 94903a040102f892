"""The oracle of MXFP4 rows (FORMAT F29): the scale by its inequality, codes by hand and by the
distance to every value, the error bound, and the unit that they make."""

import math

import numpy as np
import pytest

import oracle
from workloads import bf16_from_normal, rng_for


@pytest.mark.parametrize("amax,k", [(7.0, 0), (7.03125, 1), (3.5, -1), (6.0, 0), (1.0, -2), (0.875, -3),
                                    (2.0 ** -133, -127), (2.0 ** -126, -127), (3.3895e38, 126)])
def test_scale(amax, k):
    assert oracle.mxfp4_scale_byte(amax) == k + 127
    assert amax <= 7 * 2.0 ** k and (k == -127 or amax > 7 * 2.0 ** (k - 1))


def test_special_scales():
    assert oracle.mxfp4_scale_byte(0.0) == 127
    assert oracle.mxfp4_scale_byte(math.inf) == 255 and oracle.mxfp4_scale_byte(math.nan) == 255


def test_rounding_by_hand():
    v = [0.0, -0.0, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 6.5, 7.0, -0.25, -2.5, -7.0]
    want = [0, 8, 0, 1, 2, 2, 4, 4, 6, 6, 7, 7, 7, 8, 12, 15]
    assert list(oracle.e2m1_round(v)) == want


def test_no_element_is_off_by_more_than_half_its_step():
    x = bf16_from_normal(rng_for(910, 0), (20, 256))
    codes, scales = oracle.mxfp4_quantize(x)
    v, q = oracle.bf16_bits_to_f64(x), oracle.mxfp4_values(codes, scales)
    unit = np.repeat(np.ldexp(1.0, scales.astype(int) - 127), 32, axis=1)
    a = np.abs(v) / unit
    half = np.where(a < 2, 0.25, np.where(a < 4, 0.5, 1.0))
    assert np.all(a <= 7) and np.all(np.abs(v - q) <= half * unit)


def test_rows_make_a_unit():
    x = bf16_from_normal(rng_for(911, 0), (16, 64))
    codes, scales = oracle.mxfp4_quantize(x)
    unit = np.concatenate([oracle.mxfp4_pack(codes).reshape(-1), scales.reshape(-1)])
    assert np.array_equal(oracle.decode_mxfp4_unit(unit, 16, 64), oracle.mxfp4_values(codes, scales))
