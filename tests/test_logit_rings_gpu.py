"""The staged gradients over many rows a CTA or cluster."""
import math

import pytest
import torch

import reduction_pointwise_row_gb300 as fr

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form,rows,cols", [("persistent", 3000, 9001), ("split", 3000, 9001),
                                            ("split", 700, 90001), ("split", 200, 262145)])
def test_a_rows_place_does_not_change_its_result(form, rows, cols):
    """Equal rows at equal offsets give equal bits, whichever CTA takes them and whether
    first or later.  The ragged end is the maximum and the rest is a fifth of its half
    step in every 16-byte unit, lost when a few units at a time are added to it and not
    when all of a thread's are."""
    ld = (cols + 7) // 8 * 8
    x = torch.full((rows, ld), -math.inf, dtype=torch.bfloat16, device="cuda")
    x[:, ::8] = math.log(0.2) - 24 * math.log(2)
    x = x[:, :cols]
    x[:, cols - 1] = 0.0
    t = torch.full((rows,), cols - 1, device="cuda")
    one = torch.ones(1, device="cuda")
    z = torch.zeros(rows, 1, device="cuda")

    def matrix():
        return torch.zeros(rows, ld, dtype=x.dtype, device="cuda")[:, :cols]

    got = [fr.fr_distill_backward(x, t[:, None].contiguous(), z, one, dlogits=matrix(), form=form),
           fr.fr_xent_backward(x, t, one, dlogits=matrix(), form=form),
           {"dlogits": fr.fr_logprobs_backward(x, t, one, one, dlogits=matrix(), form=form)}]
    for n, r in enumerate(got):
        for name, v in r.items():
            others = int((v != v[:1]).reshape(rows, -1).any(1).sum())
            assert others == 0, f"call {n}, {name}: {others} of {rows} rows differ from the first"
