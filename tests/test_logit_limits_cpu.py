"""Limits of the calls over rows of logits that the host keeps, without a GPU."""
import pytest
import torch

import reduction_pointwise_row_gb300 as fr
from test_logits_cpu import OK_SO_FAR, distill, logprobs

GRID = 4 * (2 ** 31 - 1)  # rows that a grid of 4 warps a CTA has a warp for
UNSUPPORTED_FORM = 3


def test_more_rows_than_a_grid_has_warps_for():
    """Past 2^31 - 1 CTAs a launch fails, and past 2^32 their number wraps: a few rows
    would be written and the rest not.  Such calls take a form whose CTAs loop."""
    for op, many in (("logprobs", "split"), ("distill", "looped")):
        for dtype in ("bf16", "f32"):
            assert fr.fr_auto_form(op, GRID, 1, dtype, 152) == "persistent"
            for rows in (GRID + 1, 1 << 33, (1 << 34) + 8, 1 << 40):
                assert fr.fr_auto_form(op, rows, 1, dtype, 152) == many
    assert fr.fr_auto_form("logprobs", GRID, 5000, "bf16", 152) == "looped"
    assert fr.fr_auto_form("logprobs", GRID + 1, 5000, "bf16", 152) == "split"
    one = dict(cols=1, ld=1)
    for rows in (GRID + 1, (1 << 34) + 8):
        assert logprobs(rows=rows, top=1, form=1, **one) == UNSUPPORTED_FORM
        assert logprobs(rows=rows, top=0, tl=None, ti=None, form=1, **one) == UNSUPPORTED_FORM
        assert logprobs(rows=rows, top=1, form=2, **one) == UNSUPPORTED_FORM
        assert distill(rows=rows, form=1, **one) == UNSUPPORTED_FORM


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are not device memory")
def test_rows_within_the_limits_reach_the_device_check():
    one = dict(cols=1, ld=1)
    assert logprobs(rows=GRID, top=1, form=1, **one) == OK_SO_FAR
    assert distill(rows=GRID, form=1, **one) == OK_SO_FAR
    for rows in (GRID + 1, (1 << 34) + 8):
        assert logprobs(rows=rows, top=0, tl=None, ti=None, form=2, **one) == OK_SO_FAR
        assert logprobs(rows=rows, top=1, form=3, **one) == OK_SO_FAR
        assert logprobs(rows=rows, top=1, **one) == OK_SO_FAR
        assert distill(rows=rows, form=2, **one) == OK_SO_FAR


def test_bytes_of_a_gradient_without_the_entropys():
    from reduction_pointwise_row_gb300 import traffic
    count = traffic.algorithmic_bytes
    for dtype, es in (("bf16", 2), ("f32", 4)):
        assert count("logprobs_backward", 7, 1001, dtype=dtype) == 7 * (2 * es * 1001 + 16)
        assert count("logprobs_backward", 7, 1001, dtype=dtype, entropy=False) == \
            7 * (2 * es * 1001 + 12)
