"""What the binding of the residual block's calls works out before it calls the library."""
import ctypes
import math

import pytest

import reduction_pointwise_row_gb300 as fr
import rmsnorm_ref as ref


@pytest.mark.parametrize("p", [0.0, -0.0, 1e-50, 2.0**-150, 2.0**-151, 5e-324])
def test_no_dropout_where_p_is_0_in_fp32(p):
    assert ctypes.c_float(p).value == 0.0
    assert fr._rng_ptr(p, None, 0, 0) is None


@pytest.mark.parametrize("p", [math.nextafter(2.0**-150, 1.0), 2.0**-149, 1e-30, 0.5, 1.0, -1e-50, -0.5, 1.5,
                               math.nan, math.inf])
def test_a_generator_is_needed_for_any_other(p):
    with pytest.raises(ValueError):
        fr._rng_ptr(p, None, 0, 0)


def test_the_readme_advances_the_offset_past_its_sites():
    """The offset and the site are one number: sites 0 .. n - 1 of two steps share no mask where
    the offset moves by n or more, and share them all but n where it moves by 1."""
    import os
    import re
    text = open(os.path.join(os.path.dirname(__file__), "..", "README.md")).read()
    step = int(re.search(r"rng\[1\] \+= (\d+)", text).group(1))
    sites = [int(v) for v in re.findall(r"site=(\d+)", text)]
    assert sites and max(sites) < step

    def drawn(advance):
        return [{ref.keep(1, 64, 0.5, (7, k * advance), s)[0].numpy().tobytes() for s in range(step)}
                for k in (0, 1)]

    one, other = drawn(step)
    assert len(one) == len(other) == step and not one & other
    one, other = drawn(1)
    assert len(one & other) == step - 1
