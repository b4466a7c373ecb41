"""Calls one right after another on a stream: kernels may be placed while the one before
them runs, and still read what that one wrote."""
import pytest
import torch

import reduction_pointwise_row_gb300 as fr

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form,rows,cols", [("persistent", 3000, 1000), ("looped", 3000, 4097),
                                            ("split", 300, 4097), ("split", 40, 50257)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_call_reads_what_the_call_before_wrote(form, rows, cols, dtype):
    """A gradient over its logits, at once scored and distilled, many times."""
    if form == "persistent" and dtype is torch.float32:
        cols = 999
    g = torch.Generator("cuda").manual_seed(cols)
    x0 = 3 * torch.randn(rows, cols, generator=g, device="cuda", dtype=dtype)
    t = torch.randint(0, cols, (rows,), generator=g, device="cuda")
    up = 20 * torch.rand(rows, generator=g, device="cuda")
    i = torch.randint(0, cols, (rows, 8), generator=g, device="cuda")
    z = torch.randn(rows, 8, generator=g, device="cuda")
    x = x0.clone()

    def calls(sync):
        x.copy_(x0)
        sync()
        fr.fr_xent_backward(x, t, up, want_loss=False, dlogits=x)
        sync()
        r = fr.fr_logprobs(x, t, top=5, form=form)
        sync()
        # and a call behind another that only reads
        fr.fr_logprobs_backward(x, t, up, dlogits=x)
        sync()
        return [*r.values(), fr.fr_distill(x, i, z, form=form)]

    want = calls(torch.cuda.synchronize)
    runs = [calls(lambda: None) for _ in range(40)]
    for got in runs:
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert fr.fr_check_device_error() == 0
