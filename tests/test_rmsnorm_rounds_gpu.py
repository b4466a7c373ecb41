"""The norm's gradient over so many rows that every launch goes through its stages of
shared memory several times, two rows a round among them; and its sum over the rows, exactly."""
import pytest
import torch

import reduction_pointwise_row_gb300 as fr
import rmsnorm_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# (rows, cols, distance beyond cols between rows): three rounds or more of 152 CTAs without
# dropout (two rows a round up to 32 warps' units), twice as many with; rows of one to
# three units a lane, or four, that fill the warps, that do not, short ones, and rows
# that start within a unit
ROUNDS = {
    "bf16": [(60001, 128, 0), (180001, 24, 0), (60001, 72, 0), (30001, 200, 0), (12001, 1000, 0),
             (8001, 1024, 0), (9001, 768, 0), (5001, 2048, 0), (4001, 2056, 0), (2401, 4096, 0),
             (2201, 4608, 0), (1401, 8192, 0), (1401, 8184, 8), (12001, 1001, 0), (12001, 515, 2),
             (14001, 129, 0), (2401, 4097, 0), (3001, 2051, 1), (1401, 6001, 0), (2001, 4100, 0),
             (1400, 11008, 0), (1301, 13824, 0), (1401, 16384, 0)],
    "f32": [(60001, 64, 0), (60001, 60, 0), (60001, 128, 0), (20001, 256, 0), (10001, 512, 0),
            (9001, 500, 0), (5001, 1024, 0), (5001, 1020, 4), (3001, 2048, 0), (2801, 2560, 0),
            (1501, 4096, 0), (1501, 4000, 0), (9001, 509, 0), (4001, 1021, 0), (2001, 2051, 0),
            (1501, 3001, 0), (1501, 4097, 0), (1401, 6144, 0), (1401, 6000, 0), (1401, 7000, 0),
            (1401, 8192, 0)]}


def rows_of(make, rows, cols, extra, dtype):
    """A matrix whose rows lie `extra` elements further apart than they are long."""
    m = torch.zeros(rows, cols + extra, dtype=dtype, device="cuda")[:, :cols]
    m.copy_(make)
    return m


def whole(rows, cols, most, gen):
    return torch.randint(-most, most + 1, (rows, cols), generator=gen, device="cuda", dtype=torch.int8)


@pytest.mark.parametrize("dtype,rows,cols,extra", [(d, *s) for d in ROUNDS for s in ROUNDS[d]])
def test_every_stage_is_used_again(dtype, rows, cols, extra):
    """dgamma's terms are whole numbers, so that it is exact in any order: every row counts
    once.  dx of every row by the formula."""
    dt = DTYPES[dtype]
    gen = torch.Generator("cuda").manual_seed(rows + cols)
    h = rows_of(2 * whole(rows, cols, 2, gen), rows, cols, extra, dt)
    dy = rows_of(whole(rows, cols, 3, gen), rows, cols, extra, dt)
    up = rows_of(torch.randn(rows, cols, generator=gen, device="cuda"), rows, cols, extra, dt)
    gamma = 1.0 + 0.3 * torch.randn(cols, generator=gen, device="cuda")
    rstd = 0.5 * 2.0 ** torch.randint(0, 2, (rows,), generator=gen, device="cuda").float()
    n = torch.tensor([rows, cols], device="cuda")
    # at most 3 * 4 * 180001 in all: less than 2^24
    dgamma = (dy.double() * h.double() * rstd.double()[:, None]).sum(0)
    for dh in (None, up):
        d, _ = ref.backward(dy, h, gamma, rstd, dh)
        bound = ref.backward_bound(dy, h, gamma, rstd, dh, d, dt)
        for p in (0.0, 0.3):
            kw = dict(p=p, rng=n, site=1) if p else {}
            got = fr.fr_rmsnorm_backward(dy, h, gamma, rstd, dh=dh, **kw)
            assert torch.equal(got["dgamma"].double(), dgamma), f"dgamma, p {p} dh {dh is not None}"
            g = got["dresidual" if p else "dx"]
            worst = ((g.double() - d).abs() / bound).max()
            assert worst <= 1, f"p {p} dh {dh is not None}: {float(worst)} of the bound"
            if p:
                # dropout's gradient is taken before the rounding: kept elements are the
                # rounded ones times the factor within two half steps and the product's
                keep = fr.fr_dropout(torch.ones_like(h), p, n, 1) != 0
                t = ref.threshold(p)
                want = torch.where(keep, d * (65536.0 / (65536 - t)), 0.0)
                slack = bound * (65536.0 / (65536 - t)) + 2 * ref.U * want.abs()
                assert ((got["dx"].double() - want).abs() <= slack).all(), f"dx, dh {dh is not None}"
                assert (got["dx"][~keep] == 0).all()
        del d, bound


@pytest.mark.parametrize("form", ("persistent", "looped"))
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,at", [(20001, 64, 0), (3001, 1000, 1), (4001, 4097, 1), (5001, 300, 1),
                                          (3001, 8192, 0), (7001, 31, 1)])
def test_dgamma_of_the_other_forms_is_exact_too(rows, cols, at, dtype, form):
    """Element accesses (a first element off the units) and the looped form."""
    dt = DTYPES[dtype]
    gen = torch.Generator("cuda").manual_seed(rows + cols)
    h, dy = (torch.zeros(rows * cols + at, dtype=dt, device="cuda")[at:].view(rows, cols) for _ in range(2))
    h.copy_(2 * whole(rows, cols, 2, gen))
    dy.copy_(whole(rows, cols, 3, gen))
    rstd = torch.full((rows,), 0.5, device="cuda")
    got = fr.fr_rmsnorm_backward(dy, h, torch.ones(cols, device="cuda"), rstd, form=form)
    want = (dy.double() * h.double() * 0.5).sum(0)
    assert torch.equal(got["dgamma"].double(), want)
