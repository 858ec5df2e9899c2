"""Frequencies at the ends of the 64-bit range: refused where one is not finite,
and then the table stays as it was (needs no GPU)."""

import ctypes
import math

import pytest

from tensor_comm_gemm_gb300 import build as tb
from tensor_comm_gemm_gb300 import tpoverlap as t


@pytest.fixture(scope="module")
def lib():
    tb.build()
    return t.lib()


@pytest.mark.parametrize("rot,base,scaling,factor,low,high,original", [
    (8, 1e4, t.TPO_ROTARY_LINEAR, 1e-320, 1.0, 4.0, 1), (8192, 5e-324, t.TPO_ROTARY_UNSCALED, 1.0, 1.0, 4.0, 1),
    (8, 1e4, t.TPO_ROTARY_BY_PARTS, 1e-320, 1e5, 1e6, 10),
    (4, 1e-300, t.TPO_ROTARY_LINEAR, 1e-250, 1.0, 4.0, 1)])  # the second pair's only
def test_frequencies_that_are_not_finite_are_refused(lib, rot, base, scaling, factor, low, high, original):
    table = (ctypes.c_uint64 * (rot // 2))(*([7] * (rot // 2)))
    assert lib.tpo_rotary_table(rot, base, scaling, factor, low, high, original,
                                ctypes.addressof(table)) == t.TPO_ERR_INVALID_ARG
    assert "frequency" in t.tpo_last_error(), t.tpo_last_error()
    assert list(table) == [7] * (rot // 2)


@pytest.mark.parametrize("rot,base,factor", [(2, 5e-324, 1.0), (64, 1e300, 1.0), (4, 1e-300, 1.0), (64, 1e4, 1e300)])
def test_frequencies_that_are_finite_are_taken(lib, rot, base, factor):
    table = t.tpo_rotary_table(rot, base, t.TPO_ROTARY_LINEAR, factor)
    for i, got in enumerate(table.tolist()):
        turns = base ** (-2.0 * i / rot) / factor / (2 * math.pi)
        if turns < 2.0 ** 40:  # of more, few of the 53 bits are a fraction of a turn
            assert abs((got % 2 ** 64) / 2 ** 64 - turns % 1.0) <= 4 * 2.0 ** -53 * turns + 2.0 ** -63
