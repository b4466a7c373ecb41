"""What the binding of the residual block's calls works out before it calls the library."""
import ctypes
import math

import pytest

import reduction_pointwise_row_gb300 as fr


@pytest.mark.parametrize("p", [0.0, -0.0, 1e-50, 2.0**-150, 2.0**-151, 5e-324])
def test_no_dropout_where_p_is_0_in_fp32(p):
    assert ctypes.c_float(p).value == 0.0
    assert fr._rng_ptr(p, None, 0, 0) is None


@pytest.mark.parametrize("p", [math.nextafter(2.0**-150, 1.0), 2.0**-149, 1e-30, 0.5, 1.0, -1e-50, -0.5, 1.5,
                               math.nan, math.inf])
def test_a_generator_is_needed_for_any_other(p):
    with pytest.raises(ValueError):
        fr._rng_ptr(p, None, 0, 0)
