"""The norm's calls far from ordinary magnitudes: where a product of two factors of a formula
leaves fp32 and the formula's value does not."""
import math

import pytest
import torch

import reduction_pointwise_row_gb300 as fr
import rmsnorm_ref as ref
from test_rmsnorm_gpu import check_backward, check_norm, put, values, vector

pytestmark = pytest.mark.gpu

DTYPES = ("bf16", "f32")
# (cols, offset of the first element, form): the backward pass's launches -- rows of whole
# units that fill the warps and that do not, rows that start within a unit, element
# accesses, two passes
LAUNCHES = [(512, 0, "persistent"), (4096, 0, "persistent"), (1000, 0, "persistent"),
            (40, 0, "persistent"), (1003, 0, "persistent"), (1000, 1, "persistent"),
            (4096, 0, "looped"), (1003, 0, "looped")]


def scaled(rows, cols, dtype, seed, size):
    """Normal values of magnitude `size`, rounded to the type."""
    return values(rows, cols, "f32", seed).mul_(size).to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def backward(dtype, cols, at, form, size, up):
    h, dy = scaled(21, cols, dtype, 1, size), scaled(21, cols, dtype, 2, up)
    gamma = vector(cols, 30)
    rstd = ref.norm(h, gamma, 0.0)[1].float()
    got = fr.fr_rmsnorm_backward(put(dy, (at, 0)), put(h, (at, 0)), gamma.cuda(), rstd.cuda(), form=form)
    return h, dy, gamma, rstd, got


@pytest.mark.parametrize("cols,at,form", LAUNCHES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size,up", [(1e-18, 1e3), (1e16, 1e-8)])
def test_the_gradient_needs_no_square_of_rstd(size, up, dtype, cols, at, form):
    """eps 0, rstd of 1e18 and 1e-16: rstd^2 mean(u n) is past fp32 or below its normal values
    where the gradient is neither."""
    h, dy, gamma, rstd, got = backward(dtype, cols, at, form, size, up)
    check_backward(h, gamma, None, 0.0, None, 0, got, dy, rstd, f"{size} {up}")


@pytest.mark.parametrize("cols,at,form", LAUNCHES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size,up", [(1e16, 1e24), (1e-16, 1e-26)])
def test_the_gradient_needs_no_product_of_dy_and_h(size, up, dtype, cols, at, form):
    """dy h is 1e40, or 1e-42 with few bits left; dy gamma, h rstd and their product are not."""
    h, dy, gamma, rstd, got = backward(dtype, cols, at, form, size, up)
    check_backward(h, gamma, None, 0.0, None, 0, got, dy, rstd, f"{size} {up}")


@pytest.mark.parametrize("cols,at,form", LAUNCHES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size,up", [(1e-18, 1e22), (1e16, 1e-25)])
def test_dgamma_needs_no_product_of_dy_and_rstd(size, up, dtype, cols, at, form):
    """dy rstd is 1e40, or 1e-41 (as dx is, which is not looked at); dy (h rstd) is about dy."""
    h, dy, gamma, rstd, got = backward(dtype, cols, at, form, size, up)
    want = ref.backward(dy, h, gamma, rstd)[1]
    ref.assert_near(got["dgamma"], want, ref.dgamma_bound(dy, h, rstd), f"{size} {up}")


# rows held by 1-8 chunks a warp, rows in phase, element accesses, short rows, two passes
FORWARD = [(9, 1000, 0, "persistent"), (9, 1003, 0, "persistent"), (9, 1000, 1, "persistent"),
           (9, 96, 0, "persistent"), (9, 500, 0, "persistent"), (200, 512, 0, "persistent"),
           (9, 16384, 0, "persistent"), (1000, 16384, 0, "persistent"), (1300, 10240, 0, "persistent"),
           (9, 4096, 0, "looped"), (9, 1003, 0, "looped")]


@pytest.mark.parametrize("rows,cols,at,form", FORWARD)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size,weight,eps", [(1e10, 1e30, 1e-5), (1e-18, 1e-25, 0.0)])
def test_a_row_s_scale_needs_no_product_of_h_and_gamma(size, weight, eps, dtype, rows, cols, at, form):
    """h gamma is 1e40, or 1e-43 with few bits left; h rstd gamma is about gamma."""
    h, gamma = scaled(rows, cols, dtype, 3, size), vector(cols, 31) * weight
    h[1] = 0.0
    h[2] = scaled(1, cols, dtype, 4, 1.0)[0]
    h[3, cols // 2] = math.nan
    got = fr.fr_rmsnorm_quant(put(h, (at, 0)), gamma.cuda(), eps, form=form, want_rstd=True)
    y, _ = ref.norm(h, gamma, eps)
    s = got["scale"].cpu().double()[:, None]
    ref.assert_near(s, ref.scales(y, cols), (ref.rstd_bound(cols) + 4 * ref.U) * ref.scales(y, cols), "scale")
    ref.assert_near(got["y"].float().cpu().double() * s, y, ref.quant_bound(cols, y, s), "y8")


@pytest.mark.parametrize("cols,at,form", [(1000, 0, "persistent"), (1003, 0, "persistent"), (96, 0, "persistent"),
                                          (16384, 0, "persistent"), (1000, 1, "persistent"), (1003, 0, "looped")])
@pytest.mark.parametrize("dtype", DTYPES)
def test_squares_past_fp32_leave_a_row_of_zeros_in_8_bits_too(dtype, cols, at, form):
    big = torch.finfo(torch.bfloat16).max
    h = scaled(5, cols, dtype, 5, 1.0)
    h[1] = big
    gamma = vector(cols, 32).abs() + 2.0  # big gamma is past fp32
    for scale in ("row", "group"):
        got = fr.fr_rmsnorm_quant(put(h, (at, 0)), gamma.cuda(), 1e-5, scale=scale, form=form)
        assert (got["y"][1].float() == 0).all() and (got["scale"][1] == 2.0**-126).all()
        assert not got["y"].float().isnan().any() and got["scale"].isfinite().all()


@pytest.mark.parametrize("cols,at,form", [(1000, 0, "persistent"), (1003, 0, "persistent"), (96, 0, "persistent"),
                                          (16384, 0, "persistent"), (1000, 1, "persistent"), (1003, 0, "looped")])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [2.0**-126, 2.0**-127, 2.0**-129, 2.0**-149])
def test_the_smallest_given_scales(scale, dtype, cols, at, form):
    """Zeros stay zeros, NaN NaN, and the rest, far past 448 scales, the largest value."""
    x = scaled(7, cols, dtype, 6, 1.0)
    x[1] = 0.0
    x[2, 1::2] = 0.0
    x[3, 0] = math.nan
    given = torch.tensor([scale]).cuda()
    assert float(given) == scale
    y = fr.fr_rmsnorm_quant(put(x, (at, 0)), vector(cols, 33).abs().cuda(), 1e-5, scale=given,
                            form=form)["y"].float().cpu()
    want = torch.where(x == 0, 0.0, torch.copysign(torch.tensor(448.0), x.float()))
    want[3] = math.nan
    assert torch.equal(y[torch.arange(7) != 3], want[torch.arange(7) != 3]) and y[3].isnan().all()


def test_a_probability_that_rounds_to_none():
    """The calls take p in fp32: what rounds to 0 there drops nothing, as 0 does."""
    x, g = values(4, 64, "bf16", 7).cuda(), vector(64, 34).cuda()
    n = torch.tensor([1, 2], device="cuda")
    for p in (1e-50, 2.0**-151):
        assert torch.equal(fr.fr_dropout(x, p, n), x)
        assert list(fr.fr_rmsnorm(x, g, p=p, rng=n)) == ["y", "rstd"]
        rstd = fr.fr_rmsnorm(x, g)["rstd"]
        assert list(fr.fr_rmsnorm_backward(x, x, g, rstd, p=p, rng=n)) == ["dx", "dgamma"]
    got = fr.fr_rmsnorm(x, g, p=2.0**-149, rng=n)  # the smallest that does not: one of 65536
    assert "h" in got


@pytest.mark.parametrize("rows,cols", [(1000, 16384), (1200, 14336), (1500, 10496), (7400, 2048), (1900, 8192)])
def test_a_lane_adds_its_squares_in_short_runs(rows, cols):
    """A lane's first square is 1 and its others 2^-24, half a step of the sum: added to it one
    by one they would all be lost.  A lane has at most 64 squares here, of 8 chunks; added up
    in runs of 4 a term goes through 4 + 16 + 10 additions at most, of whose roundings half
    (and 4 more) reach rstd."""
    x = torch.full((rows, cols), 2.0**-12, dtype=torch.bfloat16)
    warps = -(-cols // 2048)  # of 8 chunks each, every warps-th one
    x[:, :256 * warps:8] = 1.0
    gamma = torch.ones(cols)
    want = ref.norm(x[:1], gamma, 0.0)[1].expand(rows)
    bound = ((4 + 16 + 10 + 1) / 2 + 4) * ref.U * want
    ref.assert_near(fr.fr_rmsnorm(x.cuda(), gamma.cuda(), 0.0)["rstd"], want, bound, "norm")
    got = fr.fr_rmsnorm_quant(x.cuda(), gamma.cuda(), 0.0, want_rstd=True)
    ref.assert_near(got["rstd"], want, bound, "8 bits")


@pytest.mark.parametrize("off", [1, 2, 4])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(5, 96), (33, 1000), (7, 1003), (3, 4096), (200, 768), (2, 16392)])
def test_gamma_at_any_address_in_the_forward_calls(rows, cols, dtype, off):
    x, r = values(rows, cols, dtype, 8), values(rows, cols, dtype, 9)
    gamma, n = vector(cols, 35), torch.tensor([3, 4])
    moved = torch.full((cols + 16,), math.nan, device="cuda")[off:off + cols]
    moved.copy_(gamma)
    for res, p in ((None, 0.0), (r, 0.2)):
        kw = dict(residual=None if res is None else res.cuda(), p=p, rng=n.cuda())
        check_norm(x, res, p, n, 0, fr.fr_rmsnorm(x.cuda(), moved, **kw), gamma, f"p {p}")
        for scale in ("row", "group"):
            got = fr.fr_rmsnorm_quant(x.cuda(), moved, scale=scale, **kw)
            check_norm(x, res, p, n, 0, got, gamma, f"p {p} {scale}", scale)
