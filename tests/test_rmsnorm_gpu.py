"""A residual block's row operators (fr_dropout, fr_rmsnorm, fr_rmsnorm_quant and
fr_rmsnorm_backward) against their formulas in 64 bits, at the sizes, layouts and
values where they can go wrong."""
import math
import zlib

import numpy as np
import pytest
import torch

import reduction_pointwise_row_gb300 as fr
import rmsnorm_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
# rows of one chunk and of part of one, around a chunk's and a vector's edges, several
# warps a row, every number of chunks a warp holds, the longest rows held, longer ones
SHAPES = [(1, 1), (3, 7), (5, 8), (9, 31), (300, 64), (33, 100), (7, 255), (7, 256), (5, 257),
          (65, 512), (11, 520), (200, 768), (33, 1000), (400, 1025), (4, 2056), (3, 4097),
          (160, 5120), (2, 8192), (3, 8199), (3, 8200), (305, 8448), (2, 16383), (3, 16384),
          (2, 16392), (2, 20001), (1, 70000)]
# offset of the first element and distance beyond cols between rows, in elements
LAYOUTS = [(0, 0), (8, 16), (1, 0), (0, 3)]
GUARD = 0x5A


def gen(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def values(rows, cols, dtype, seed, std=1.0):
    return torch.randn(rows, cols, generator=gen(rows, cols, seed)).mul_(std).to(DTYPES[dtype])


def vector(n, seed):
    return 1.0 + 0.3 * torch.randn(n, generator=gen(n, seed))


def rng_of(seed):
    return torch.randint(-2**63, 2**63 - 1, (2,), generator=gen("rng", seed))


class Placed:
    """A matrix on the GPU within a buffer whose other bytes must stay as they are."""

    def __init__(self, rows, cols, dtype, offset=0, extra=0):
        es = torch.empty(0, dtype=dtype).element_size()
        ld, self.es = cols + extra, es
        self.raw = torch.full(((offset + rows * ld + 64) * es,), GUARD, dtype=torch.uint8, device="cuda")
        self.t = self.raw.view(dtype).as_strided((rows, cols), (ld, 1), offset)
        self.free = torch.ones(self.raw.numel(), dtype=torch.bool)
        self.free.as_strided((rows, cols * es), (ld * es, 1), offset * es).fill_(False)

    def intact(self):
        return bool((self.raw.cpu()[self.free] == GUARD).all())


def put(x, layout=(0, 0)):
    p = Placed(*x.shape, x.dtype, *layout)
    p.t.copy_(x)
    return p.t


def out(x, layout=(0, 0), dtype=None):
    return Placed(*x.shape, dtype or x.dtype, *layout)


def skip_long(form, cols, backward=False, dtype="bf16", layout=(0, 0)):
    most = 16384
    if backward and (dtype == "f32" or cols % 8 or any(v % 8 for v in layout)):
        most = 8192
    if form == "persistent" and cols > most:
        pytest.skip("a row longer than a CTA's registers")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_dropout_shapes(rows, cols, dtype):
    x, r = values(rows, cols, dtype, 1), values(rows, cols, dtype, 2, 2.0)
    n = rng_of(cols)
    for i, layout in enumerate(LAYOUTS):
        p = (0.1, 0.5, 0.0, 1.0)[i]
        for res in (None, r):
            o = out(x, layout)
            fr.fr_dropout(put(x, layout), p, n.cuda(), i, out=o.t,
                          residual=None if res is None else put(res, LAYOUTS[i - 1]))
            want = ref.dropout(x, p, n, i, res)
            ref.assert_near(o.t, want, ref.dropout_bound(x, p, res, want, DTYPES[dtype]),
                            f"{layout} {p}")
            assert o.intact()


def check_norm(x, res, p, n, site, got, gamma, what, quant=None, given=None):
    """The outputs in `got` against the formulas; y's of the h that came back."""
    dtype, cols = x.dtype, x.shape[1]
    h = x
    if p or res is not None:
        want = ref.dropout(x, p, n, site, res)
        ref.assert_near(got["h"], want, ref.dropout_bound(x, p, res, want, dtype), f"{what} h")
        h = got["h"].cpu()
    else:
        assert "h" not in got
    y, rstd = ref.norm(h, gamma, EPS)
    if "rstd" in got:
        ref.assert_near(got["rstd"], rstd, ref.rstd_bound(cols) * rstd, f"{what} rstd")
    if quant is None:
        ref.assert_near(got["y"], y, ref.norm_bound(cols, y, dtype), f"{what} y")
        return
    if quant == "given":
        s = given.double().expand(x.shape[0], 1)
        assert "scale" not in got
    else:
        width = cols if quant == "row" else fr.SCALE_COLS
        want = ref.scales(y, width)
        s = got["scale"].cpu().double().view(want.shape)
        ref.assert_near(s, want, (ref.rstd_bound(cols) + 4 * ref.U) * want, f"{what} scale")
    s = s.repeat_interleave(fr.SCALE_COLS, 1)[:, :cols] if quant == "group" else s.expand(y.shape)
    v = y.clamp(-448.0 * s, 448.0 * s)
    ref.assert_near(got["y"].float().cpu().double() * s, v, ref.quant_bound(cols, v, s), f"{what} y8")


@pytest.mark.parametrize("form", ("persistent", "looped"))
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_rmsnorm_shapes(rows, cols, dtype, form):
    skip_long(form, cols)
    x, r = values(rows, cols, dtype, 3), values(rows, cols, dtype, 4, 3.0)
    gamma, n = vector(cols, 1), rng_of(cols + 1)
    for i, layout in enumerate(LAYOUTS):
        for res, p in ((None, 0.0), (r, 0.0), (r, 0.2), (None, 0.5)):
            what = f"{layout} p {p} residual {res is not None}"
            y, kw = out(x, layout), {}
            if p or res is not None:
                h = out(x, LAYOUTS[(i + 1) % 4] if i else layout)
                kw = dict(h=h.t, p=p, rng=n.cuda(), site=i,
                          residual=None if res is None else put(res, layout))
            got = fr.fr_rmsnorm(put(x, layout), gamma.cuda(), EPS, form=form, out=y.t, **kw)
            assert fr.fr_last_form() == form
            check_norm(x, res, p, n, i, got, gamma, what)
            assert y.intact() and (not kw or h.intact()), what


@pytest.mark.parametrize("form", ("persistent", "looped"))
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_rmsnorm_quant_shapes(rows, cols, dtype, form):
    skip_long(form, cols)
    x, r = values(rows, cols, dtype, 5), values(rows, cols, dtype, 6, 3.0)
    gamma, n = vector(cols, 2), rng_of(cols + 2)
    given = torch.tensor([0.004])  # many values past 448 of them
    groups = -(-cols // fr.SCALE_COLS)
    for i, layout in enumerate(LAYOUTS):
        for quant in ("row", "group", "given"):
            res, p = ((None, 0.0), (r, 0.0), (r, 0.2), (None, 0.5))[(i + len(quant)) % 4]
            y, kw = out(x, layout, torch.float8_e4m3fn), {}
            if p or res is not None:
                kw = dict(p=p, rng=n.cuda(), site=i, residual=None if res is None else put(res, layout))
            if quant == "group" and i % 2:  # one group's scales of all rows together
                kw["scale_out"] = torch.empty(groups, rows, device="cuda").t()
            got = fr.fr_rmsnorm_quant(put(x, layout), gamma.cuda(), EPS, form=form, out=y.t,
                                      scale=given.cuda() if quant == "given" else quant,
                                      want_rstd=i == 0, **kw)
            assert got["y"].dtype == torch.float8_e4m3fn and ("rstd" in got) == (i == 0)
            check_norm(x, res, p, n, i, got, gamma, f"{layout} {quant} p {p}", quant, given)
            assert y.intact()


def check_backward(x, gamma, dh, p, n, site, got, dy, rstd, what):
    d, dgamma = ref.backward(dy, x, gamma, rstd, dh)
    b = ref.backward_bound(dy, x, gamma, rstd, dh, d, x.dtype)
    if p:
        if "dresidual" in got:
            ref.assert_near(got["dresidual"], d, b, f"{what} dresidual")
        m, f = ref.keep(*x.shape, p, n, site)
        d, b = torch.where(m, d * f, 0.0), torch.where(m, b * f + 2 * ref.U * d.abs() * f, 0.0)
    else:
        assert "dresidual" not in got
    ref.assert_near(got["dx"], d, b, f"{what} dx")
    if "dgamma" in got:
        ref.assert_near(got["dgamma"], dgamma, ref.dgamma_bound(dy, x, rstd), f"{what} dgamma")


@pytest.mark.parametrize("form", ("persistent", "looped"))
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward_shapes(rows, cols, dtype, form):
    x, dy, up = (values(rows, cols, dtype, 7 + i, s) for i, s in enumerate((2.0, 0.1, 0.1)))
    gamma, n = vector(cols, 3), rng_of(cols + 3)
    rstd = ref.norm(x, gamma, EPS)[1].float()
    done = 0
    for i, layout in enumerate(LAYOUTS):
        if form == "persistent" and cols > (8192 if dtype == "f32" or cols % 8 or i > 1 else 16384):
            continue
        done += 1
        for dh, p in ((None, 0.0), (up, 0.0), (up, 0.2), (None, 0.5)):
            what = f"{layout} p {p} dh {dh is not None}"
            dx, kw = out(x, layout), {}
            if p:
                dr = out(x, layout)
                kw = dict(p=p, rng=n.cuda(), site=i, dresidual=dr.t)
            got = fr.fr_rmsnorm_backward(put(dy, layout), put(x, LAYOUTS[i - 1] if i > 1 else layout),
                                         gamma.cuda(), rstd.cuda(), form=form, dx=dx.t,
                                         dh=None if dh is None else put(dh, layout), **kw)
            assert fr.fr_last_form() == form
            check_backward(x, gamma, dh, p, n, i, got, dy, rstd, what)
            assert dx.intact() and (not p or dr.intact()), what
    if not done:
        pytest.skip("a row longer than a CTA's registers")


@pytest.mark.parametrize("rows,cols", [(20000, 64), (5000, 768), (3001, 1000), (2500, 4096),
                                       (1500, 4097), (1400, 8192), (700, 16384)])
def test_many_rows(rows, cols):
    """More rows than CTAs at once: every CTA takes several."""
    x, r, dy = (values(rows, cols, "bf16", 20 + i) for i in range(3))
    gamma, n = vector(cols, 4), rng_of(9)
    xc, nc = x.cuda(), n.cuda()
    got = fr.fr_rmsnorm(xc, gamma.cuda(), EPS, residual=r.cuda(), p=0.1, rng=nc, site=2)
    check_norm(x, r, 0.1, n, 2, got, gamma, "forward")
    h = got["h"].cpu()
    back = fr.fr_rmsnorm_backward(dy.cuda(), got["h"], gamma.cuda(), got["rstd"], dh=xc, p=0.1, rng=nc,
                                  site=2)
    check_backward(h, gamma, x, 0.1, n, 2, back, dy, got["rstd"].cpu(), "backward")
    q = fr.fr_rmsnorm_quant(got["h"], gamma.cuda(), EPS, scale="group")
    check_norm(h, None, 0.0, n, 0, q, gamma, "quant", "group")


@pytest.mark.parametrize("form", ("persistent", "looped"))
@pytest.mark.parametrize("cols", [96, 1003, 4096])
def test_special_values(cols, form):
    """Rows of zeros, of NaN, infinities, the type's extremes and subnormals, beside
    ordinary ones, which they leave alone."""
    x = values(9, cols, "bf16", 30)
    gamma = vector(cols, 5)
    big = torch.finfo(torch.bfloat16).max
    x[1] = 0.0
    x[2, cols // 2] = math.nan
    x[3, 0] = math.inf
    x[4, cols - 1] = -math.inf
    x[5] = big  # its squares add up past fp32: rstd 0
    x[6] = 1e-30
    x[7] = 0.0
    x[7, 3] = 2.0 ** -100
    plain = torch.tensor([0, 1, 6, 7, 8])
    got = fr.fr_rmsnorm(x.cuda(), gamma.cuda(), EPS, form=form)
    y, rstd = (got[k].cpu() for k in ("y", "rstd"))
    wy, wr = ref.norm(x, gamma, EPS)
    ref.assert_near(rstd[plain], wr[plain], ref.rstd_bound(cols) * wr[plain], "rstd")
    ref.assert_near(y[plain], wy[plain], ref.norm_bound(cols, wy[plain], torch.bfloat16), "y")
    assert y[2].isnan().all() and rstd[2].isnan()
    for r, at in ((3, 0), (4, cols - 1)):
        others = torch.arange(cols) != at
        assert rstd[r] == 0 and y[r, at].isnan() and (y[r, others] == 0).all()
    assert rstd[5] == 0 and (y[5] == 0).all()
    for scale in ("row", "group"):
        q = fr.fr_rmsnorm_quant(x.cuda(), gamma.cuda(), EPS, scale=scale, form=form)
        y8, s = q["y"].float().cpu(), q["scale"].cpu().view(9, -1)
        assert (y8[1] == 0).all() and (s[1] == 2.0 ** -126).all()
        assert y8[2].isnan().all() and s[2].isnan().all()
        whole = range(cols) if scale == "row" else range(128)
        assert y8[3, list(whole)[:cols]].isnan().all() and s[3, 0].isnan()
        assert s[8].isfinite().all() and not y8[8].isnan().any()
        for r in (0, 6, 8):
            v = wy[r:r + 1]
            sc = s[r:r + 1].double()
            sc = sc.repeat_interleave(128, 1)[:, :cols] if scale == "group" else sc.expand(1, cols)
            ref.assert_near(y8[r:r + 1].double() * sc, v, ref.quant_bound(cols, v, sc), f"{scale} {r}")
    # eps 0: a row of zeros has no direction
    zero = fr.fr_rmsnorm(x.cuda(), gamma.cuda(), 0.0, form=form)
    assert zero["y"][1].isnan().all() and not zero["y"][0].isnan().any()
    # the backward pass: a NaN row gives itself and dgamma NaN, and no other row
    dy = values(9, cols, "bf16", 31)
    back = fr.fr_rmsnorm_backward(dy.cuda(), x.cuda(), gamma.cuda(), got["rstd"], form=form)
    dx = back["dx"].cpu()
    assert dx[2].isnan().all() and back["dgamma"].isnan().all()
    for r in (0, 1, 6, 8):
        sl = slice(r, r + 1)
        d, _ = ref.backward(dy[sl], x[sl], gamma, rstd[sl])
        ref.assert_near(dx[sl], d, ref.backward_bound(dy[sl], x[sl], gamma, rstd[sl], None, d, x.dtype),
                        f"row {r}")


@pytest.mark.parametrize("cols", [512, 1003, 20000])
def test_dropped_elements_may_hold_anything(cols):
    """What is dropped is 0, and its gradient 0, whatever it holds."""
    rows, p, n = 40, 0.5, rng_of(3)
    m, _ = ref.keep(rows, cols, p, n, 1)
    x = values(rows, cols, "f32", 40)
    bad = x.clone()
    bad[~m] = torch.tensor([math.nan, math.inf, -math.inf]).repeat(rows * cols)[:int((~m).sum())]
    gamma, nc = vector(cols, 6).cuda(), n.cuda()
    assert torch.equal(fr.fr_dropout(bad.cuda(), p, nc, 1), fr.fr_dropout(x.cuda(), p, nc, 1))
    a, b = (fr.fr_rmsnorm(v.cuda(), gamma, p=p, rng=nc, site=1) for v in (x, bad))
    assert all(torch.equal(a[k], b[k]) for k in a)
    r = values(rows, cols, "f32", 41).cuda()
    gone = fr.fr_dropout(bad.cuda(), 1.0, nc, 1, residual=r)
    assert torch.equal(gone, r)
    d = fr.fr_rmsnorm_backward(r, a["h"], gamma, a["rstd"], p=p, rng=nc, site=1)
    assert (d["dx"].cpu()[~m] == 0).all() and (d["dresidual"].cpu()[~m] != 0).any()
    assert torch.equal(d["dx"].cpu() != 0, m & (d["dresidual"].cpu() != 0))


def test_the_mask_does_not_depend_on_layout_type_or_call():
    """One mask for a place in the model: whatever the alignment, the type, the form, the
    call that draws it, and the seed's and offset's sign."""
    rows, cols, p = 50, 1000, 0.3
    for n in (torch.tensor([-1, -5]), torch.tensor([1 << 40, (1 << 32) - 2]), rng_of(5)):
        m, _ = ref.keep(rows, cols, p, n, 7)
        nc = n.cuda()
        for dtype in DTYPES:
            one = torch.ones(rows, cols, dtype=DTYPES[dtype])
            for layout in LAYOUTS:
                v = put(one, layout)
                masks = [fr.fr_dropout(v, p, nc, 7) != 0]
                for form in ("persistent", "looped"):
                    masks.append(fr.fr_rmsnorm(v, torch.ones(cols, device="cuda"), p=p, rng=nc, site=7,
                                               form=form)["h"] != 0)
                    masks.append(fr.fr_rmsnorm_backward(
                        v, put(torch.zeros_like(one)), torch.ones(cols, device="cuda"),
                        torch.ones(rows, device="cuda"), p=p, rng=nc, site=7, form=form)["dx"] != 0)
                for k in masks:
                    assert torch.equal(k.cpu(), m)
    a = fr.fr_dropout(v, p, (nc + torch.tensor([0, 7], device="cuda")), 0)
    assert torch.equal(a, fr.fr_dropout(v, p, nc, 7))


def block(x, r, gamma, dy, n, site=0, p=0.1):
    """A training step's row work of a block, and an 8-bit forward pass beside it."""
    a = fr.fr_rmsnorm(x, gamma, EPS, residual=r, p=p, rng=n, site=site)
    b = fr.fr_rmsnorm_backward(dy, a["h"], gamma, a["rstd"], dh=dy, p=p, rng=n, site=site)
    q = fr.fr_rmsnorm_quant(a["y"], gamma, EPS, scale="group", residual=a["h"])
    d = fr.fr_dropout(b["dx"], p, n, site + 1, residual=b["dresidual"])
    return [a["y"], a["h"], a["rstd"], b["dx"], b["dresidual"], b["dgamma"], q["y"].view(torch.uint8),
            q["scale"], q["h"], d]


def test_a_block_as_it_is_used():
    """The calls together: the norm's sum is fr_dropout's, its gradient agrees with
    differences of the forward pass, and the 8-bit output with the other."""
    rows, cols, p, site = 6, 130, 0.25, 4
    x, r, dy, dh = (values(rows, cols, "f32", 50 + i) for i in range(4))
    gamma, n = vector(cols, 7), rng_of(11)
    nc, gc = n.cuda(), gamma.cuda()
    a = fr.fr_rmsnorm(x.cuda(), gc, EPS, residual=r.cuda(), p=p, rng=nc, site=site)
    assert torch.equal(a["h"], fr.fr_dropout(x.cuda(), p, nc, site, residual=r.cuda()))
    plain = fr.fr_rmsnorm(a["h"], gc, EPS)
    assert torch.equal(plain["y"], a["y"]) and torch.equal(plain["rstd"], a["rstd"])
    b = fr.fr_rmsnorm_backward(dy.cuda(), a["h"], gc, a["rstd"], dh=dh.cuda(), p=p, rng=nc, site=site)
    assert torch.equal(b["dx"], fr.fr_dropout(b["dresidual"], p, nc, site))

    m, f = ref.keep(rows, cols, p, n, site)

    def loss(x, r, gamma):
        h = r + torch.where(m, x * f, 0.0)
        return float((ref.norm(h, gamma, EPS)[0] * dy.double()).sum() + (h * dh.double()).sum())

    step = 1e-4
    at = [x.double(), r.double(), gamma.double()]
    pick = gen("pick")
    for which, grad in enumerate((b["dx"], b["dresidual"], b["dgamma"])):
        for k in torch.randint(0, grad.numel(), (12,), generator=pick).tolist():
            lo, hi = ([v.clone() for v in at] for _ in range(2))
            lo[which].view(-1)[k] -= step
            hi[which].view(-1)[k] += step
            slope = (loss(*hi) - loss(*lo)) / (2 * step)
            # differences are off by step^2 times a third derivative (of order 1 to 10 here)
            # and the loss's rounding (2^-53 of about 100) / step
            assert abs(float(grad.view(-1)[k]) - slope) < 1e-5 * max(1.0, abs(slope)), (which, k)

    q = fr.fr_rmsnorm_quant(x.cuda(), gc, EPS, scale="row", residual=r.cuda(), p=p, rng=nc, site=site)
    assert torch.equal(q["h"], a["h"])
    y = a["y"].cpu().double()
    s = q["scale"].cpu().double()[:, None]
    ref.assert_near(q["y"].float().cpu().double() * s, y,
                    ref.quant_bound(cols, y, s) + 2 * ref.norm_bound(cols, y, torch.float32), "8 bits")


@pytest.mark.parametrize("rows,cols", [(1, 8192), (37, 4097), (300, 4096), (6, 20000)])
def test_captured_replayed_and_on_other_streams(rows, cols):
    """A captured graph's replay on new data and a new seed, two graphs replayed at once on
    two streams, and a call on a side stream give what eager calls give."""
    def data(seed):
        return [*(values(rows, cols, "bf16", 60 + seed + i).cuda() for i in (0, 1)),
                vector(cols, seed).cuda(), values(rows, cols, "bf16", 70 + seed).cuda(),
                rng_of(seed).cuda()]

    graphs = []
    for seed in (1, 2):
        held = data(seed)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            block(*held)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = block(*held)
        graphs.append((g, held, outs))
    for (_, held, _), seed in zip(graphs, (3, 4)):
        for h, v in zip(held, data(seed)):
            h.copy_(v)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for (g, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, held, outs in graphs:
        want = block(*held)
        torch.cuda.synchronize()
        for o, e in zip(outs, want):
            assert torch.equal(o, e)
    x, r, gamma, dy, n = data(9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = fr.fr_rmsnorm(x, gamma, residual=r, p=0.1, rng=n, stream=s)
    b = fr.fr_rmsnorm_backward(dy, a["h"], gamma, a["rstd"], p=0.1, rng=n, stream=s)
    q = fr.fr_rmsnorm_quant(x, gamma, stream=s)
    d = fr.fr_dropout(x, 0.5, n, stream=s)
    s.synchronize()
    a2 = fr.fr_rmsnorm(x, gamma, residual=r, p=0.1, rng=n)
    b2 = fr.fr_rmsnorm_backward(dy, a["h"], gamma, a["rstd"], p=0.1, rng=n)
    assert torch.equal(a["y"], a2["y"]) and torch.equal(b["dx"], b2["dx"])
    assert torch.equal(b["dgamma"], b2["dgamma"])
    assert torch.equal(q["scale"], fr.fr_rmsnorm_quant(x, gamma)["scale"])
    assert torch.equal(d, fr.fr_dropout(x, 0.5, n))


@pytest.mark.parametrize("rows,cols", [(1, 512), (700, 1000), (333, 8192), (400, 4097), (20, 17000)])
def test_runs_repeat_bit_for_bit(rows, cols):
    args = [values(rows, cols, "bf16", 80).cuda(), values(rows, cols, "bf16", 81).cuda(),
            vector(cols, 8).cuda(), values(rows, cols, "bf16", 82).cuda(), rng_of(8).cuda()]
    first = [o.clone() for o in block(*args)]
    for _ in range(5):
        for o, f in zip(block(*args), first):
            assert torch.equal(o, f)


@pytest.mark.parametrize("form", ("persistent", "looped"))
@pytest.mark.parametrize("cols", [768, 1003, 4096])
def test_outputs_in_the_inputs_buffers(cols, form):
    rows = 400
    x, r, dy, dh = (values(rows, cols, "bf16", 90 + i).cuda() for i in range(4))
    gamma, n = vector(cols, 9).cuda(), rng_of(2).cuda()
    kw = dict(p=0.1, rng=n, site=1, form=form)
    want = fr.fr_rmsnorm(x, gamma, EPS, residual=r, **kw)
    for h, y in (("r", "x"), ("x", "r"), ("r", None), ("x", None)):
        b = {"x": x.clone(), "r": r.clone(), None: torch.empty_like(x)}
        got = fr.fr_rmsnorm(b["x"], gamma, EPS, residual=b["r"], h=b[h], out=b[y], **kw)
        assert all(torch.equal(got[k], want[k]) for k in want), (h, y)
    v = x.clone()
    assert torch.equal(fr.fr_rmsnorm(v, gamma, EPS, out=v, form=form)["y"],
                       fr.fr_rmsnorm(x, gamma, EPS, form=form)["y"])
    q = fr.fr_rmsnorm_quant(x, gamma, EPS, residual=r, **kw)
    b = r.clone()
    q2 = fr.fr_rmsnorm_quant(x, gamma, EPS, residual=b, h=b, **kw)
    assert torch.equal(q2["h"], q["h"]) and torch.equal(q2["scale"], q["scale"])
    for o in ("x", "r"):
        b = {"x": x.clone(), "r": r.clone()}
        fr.fr_dropout(b["x"], 0.1, n, 1, residual=b["r"], out=b[o])
        assert torch.equal(b[o], want["h"])
    w = fr.fr_rmsnorm_backward(dy, want["h"], gamma, want["rstd"], dh=dh, **kw)
    for one, two in (("dy", "h"), ("h", "dh"), ("dh", "dy")):
        b = {"dy": dy.clone(), "h": want["h"].clone(), "dh": dh.clone()}
        got = fr.fr_rmsnorm_backward(b["dy"], b["h"], gamma, want["rstd"], dh=b["dh"], dx=b[one],
                                     dresidual=b[two], **kw)
        assert all(torch.equal(got[k], w[k]) for k in w), (one, two)
    # the two halves of one buffer: each in the gaps of the other
    both = torch.empty(rows, 2 * cols, dtype=x.dtype, device="cuda")
    both[:, :cols] = x
    got = fr.fr_rmsnorm(both[:, :cols], gamma, EPS, out=both[:, cols:], form=form)
    # (another alignment adds up a row's squares in another order: not the same bits)
    check_norm(x.cpu(), None, 0.0, None, 0, got, gamma.cpu(), "gaps")
    assert torch.equal(both[:, :cols], x)


def test_row_offsets_past_32_bits():
    """Rows whose elements lie past 2^32 bytes and 2^31 elements of their base."""
    cols, ld = 1008, (1 << 31) + 24
    buf = torch.empty(2 * ld + 2 * cols, dtype=torch.bfloat16, device="cuda")
    far = buf.as_strided((3, cols), (ld, 1), 0)
    x, r = values(3, cols, "bf16", 100), values(3, cols, "bf16", 101)
    gamma, n = vector(cols, 10), rng_of(4)
    for shift in (0, 1):
        v = buf.as_strided((3, cols), (ld, 1), shift)
        for form in ("persistent", "looped"):
            v.copy_(x)
            got = fr.fr_rmsnorm(v, gamma.cuda(), EPS, residual=r.cuda(), h=v, p=0.1, rng=n.cuda(),
                                form=form)
            check_norm(x, r, 0.1, n, 0, got, gamma, f"{form} {shift}")
            h = v.cpu()
            back = fr.fr_rmsnorm_backward(v, v, gamma.cuda(), got["rstd"], dx=v, form=form)
            check_backward(h, gamma, None, 0.0, n, 0, back, h, got["rstd"].cpu(), f"{form} {shift}")
        v.copy_(x)
        fr.fr_dropout(v, 0.3, n.cuda(), out=v)
        want = ref.dropout(x, 0.3, n)
        ref.assert_near(v, want, ref.dropout_bound(x, 0.3, None, want, x.dtype))
    del far


def test_outputs_that_are_not_wanted_and_given_ones():
    x, dy = values(33, 520, "bf16", 110).cuda(), values(33, 520, "bf16", 111).cuda()
    gamma, n = vector(520, 11).cuda(), rng_of(1).cuda()
    full = fr.fr_rmsnorm(x, gamma)
    assert list(fr.fr_rmsnorm(x, gamma, want_rstd=False)) == ["y"]
    rstd, h = torch.empty(33, device="cuda"), torch.empty_like(x)
    got = fr.fr_rmsnorm(x, gamma, rstd=rstd, want_rstd=False)
    assert got["rstd"] is rstd and torch.equal(rstd, full["rstd"])
    got = fr.fr_rmsnorm_quant(x, gamma, residual=dy, h=h, rstd=rstd)
    assert got["h"] is h and got["rstd"] is rstd
    kw = dict(p=0.2, rng=n)
    all_ = fr.fr_rmsnorm_backward(dy, x, gamma, full["rstd"], **kw)
    for a, b in ((False, True), (True, False), (False, False)):
        got = fr.fr_rmsnorm_backward(dy, x, gamma, full["rstd"], want_dgamma=a, want_dresidual=b, **kw)
        assert ("dgamma" in got, "dresidual" in got) == (a, b)
        assert all(torch.equal(got[k], all_[k]) for k in got)
    dg = torch.empty(520, device="cuda")
    nws = fr.fr_workspace_size("rmsnorm_backward", 33, 520, "bf16")
    ws = torch.full((nws + 64,), GUARD, dtype=torch.uint8, device="cuda")
    got = fr.fr_rmsnorm_backward(dy, x, gamma, full["rstd"], dgamma=dg, workspace=ws[:nws], **kw)
    assert got["dgamma"] is dg and torch.equal(dg, all_["dgamma"])
    assert (ws[nws:] == GUARD).all()
    with pytest.raises(fr.FRError):
        fr.fr_rmsnorm_backward(dy, x, gamma, full["rstd"], workspace=ws[:nws - 4], **kw)


def test_the_binding_refuses():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    g, n = torch.ones(64, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    s, r = torch.ones(4, device="cuda"), torch.ones_like(x)
    bad = [
        lambda: fr.fr_dropout(x.half(), 0.5, n), lambda: fr.fr_dropout(x, 1.5, n),
        lambda: fr.fr_dropout(x, -0.5, n), lambda: fr.fr_dropout(x, 0.5, None),
        lambda: fr.fr_dropout(x, 0.5, n.int()), lambda: fr.fr_dropout(x, 0.5, n.cpu()),
        lambda: fr.fr_dropout(x, 0.5, n[:1]), lambda: fr.fr_dropout(x, 0.5, n.repeat(2)[::2]),
        lambda: fr.fr_dropout(x, 0.5, n, 1 << 63), lambda: fr.fr_dropout(x, math.nan, n),
        lambda: fr.fr_dropout(x, 0.5, n, residual=x.float()),
        lambda: fr.fr_dropout(x, 0.5, n, out=x[:, :32]), lambda: fr.fr_dropout(x[:0], 0.5, n),
        lambda: fr.fr_dropout(x, 0.5, n, out=torch.zeros(4, 128, device="cuda").bfloat16()[:, ::2]),
        lambda: fr.fr_rmsnorm(x, g[:32]), lambda: fr.fr_rmsnorm(x, g.bfloat16()),
        lambda: fr.fr_rmsnorm(x, g.repeat(2)[::2]), lambda: fr.fr_rmsnorm(x, g, h=r),
        lambda: fr.fr_rmsnorm(x, g, p=0.5), lambda: fr.fr_rmsnorm(x, g, residual=r, h=r.float()),
        lambda: fr.fr_rmsnorm(x, g, rstd=s[:3]), lambda: fr.fr_rmsnorm(x, g, out=x.float()),
        lambda: fr.fr_rmsnorm_quant(x, g, scale="column"), lambda: fr.fr_rmsnorm_quant(x, g, scale=s),
        lambda: fr.fr_rmsnorm_quant(x, g, scale=s[:1].double()),
        lambda: fr.fr_rmsnorm_quant(x, g, scale=s[:1], scale_out=s),
        lambda: fr.fr_rmsnorm_quant(x, g, scale_out=s[:3]), lambda: fr.fr_rmsnorm_quant(x, g, out=r),
        lambda: fr.fr_rmsnorm_backward(x, r[:3], g, s), lambda: fr.fr_rmsnorm_backward(x, r, g, s[:3]),
        lambda: fr.fr_rmsnorm_backward(x, r, g, s, dresidual=r.clone()),
        lambda: fr.fr_rmsnorm_backward(x, r, g, s, dh=r.float()),
        lambda: fr.fr_rmsnorm_backward(x, r, g, s, dgamma=s),
        lambda: fr.fr_rmsnorm_backward(x, r, g, s, workspace=torch.empty(64)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("accepted", i)
    wide = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: fr.fr_rmsnorm(x, g, -1.0), lambda: fr.fr_rmsnorm(x, g, math.inf),
                 lambda: fr.fr_rmsnorm(x, g, residual=r, h=x, out=x),
                 lambda: fr.fr_rmsnorm(wide[:, :64], g, out=wide[:, 63:127]),
                 lambda: fr.fr_rmsnorm(x, g, form="split"),
                 lambda: fr.fr_rmsnorm_quant(x, g, out=x.view(torch.float8_e4m3fn)[:, :64]),
                 lambda: fr.fr_rmsnorm_backward(x, r, g, s, form="split"),
                 lambda: fr.fr_rmsnorm_backward(x, r, g, s, dgamma=g)):
        with pytest.raises(fr.FRError):
            call()
    long = torch.zeros(1, 16392, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fr.FRError):
        fr.fr_rmsnorm(long, torch.ones(16392, device="cuda"), form="persistent")


def test_single_columns_rows_and_groups_in_either_order():
    """Strides of dimensions of one element do not count."""
    for rows, cols in ((1, 300), (5, 100), (1, 64), (5, 1)):
        x, gamma = values(rows, cols, "bf16", 120), vector(cols, 12)
        groups = -(-cols // 128)
        for so in (torch.empty(rows, groups, device="cuda"), torch.empty(groups, rows, device="cuda").t()):
            got = fr.fr_rmsnorm_quant(x.cuda(), gamma.cuda(), EPS, scale="group", scale_out=so)
            check_norm(x, None, 0.0, None, 0, got, gamma, f"{rows}x{cols}", "group")
    spaced = torch.full((10,), -1.0, device="cuda")
    x = values(5, 64, "bf16", 121)
    got = fr.fr_rmsnorm_quant(x.cuda(), torch.ones(64, device="cuda"), EPS, scale_out=spaced[::2])
    check_norm(x, None, 0.0, None, 0, got, torch.ones(64), "spaced", "row")
    assert (spaced[1::2] == -1.0).all()
    one = torch.ones(5, 1)
    y = fr.fr_rmsnorm(one.cuda(), torch.ones(1, device="cuda"), 0.0)["y"]
    assert torch.equal(y.cpu(), one)


def test_another_device_is_refused():
    x = torch.zeros(2, 8, device="cuda")

    class Far(torch.Tensor):
        def get_device(self):
            return torch.cuda.current_device() + 1

    g = torch.ones(8, device="cuda").as_subclass(Far)
    with pytest.raises(ValueError, match="current device"):
        fr.fr_rmsnorm(x, g)


def test_numpy_and_torch_agree_on_the_bits():
    """The mask's words, bit for bit, at a far row and block."""
    n = np.array([0x0123456789ABCDEF, 0x7FFFFFFFFFFFFFFF])
    rows, cols = 3, 70001
    m, _ = ref.keep(rows, cols, 0.5, n, 1)  # the offset wraps past the largest int64
    got = fr.fr_dropout(torch.ones(rows, cols, device="cuda"), 0.5, torch.from_numpy(n).cuda(), 1)
    assert torch.equal(got.cpu() != 0, m)


# Row lengths of each launch of the backward pass's ring: one to four units a lane, exact
# ones (whole units of every lane) and others, one to sixteen warps a row; strides of each
# class of phases; fewer rows than classes and than row groups, and several rounds.
RINGS = {"bf16": [(900, 8, 0), (1900, 72, 0), (700, 128, 8), (1300, 256, 0), (650, 264, 0),
                  (640, 768, 0), (641, 769, 0), (500, 1024, 0), (310, 1030, 2), (311, 1500, 4),
                  (400, 2048, 0), (333, 2051, 1), (330, 4098, 6), (500, 4100, 0), (320, 4352, 0),
                  (5, 4097, 0), (9, 515, 0), (317, 5120, 0), (312, 5121, 7), (306, 8186, 6),
                  (308, 8192, 0), (155, 9216, 0), (160, 16384, 0), (153, 10000, 0),
                  (310, 5376, 0), (160, 8200, 0), (155, 11008, 0), (154, 12288, 0), (157, 13824, 8)],
         "f32": [(900, 4, 0), (1000, 60, 0), (700, 130, 2), (640, 512, 0), (620, 516, 0),
                 (610, 517, 0), (400, 1024, 4), (333, 2050, 0), (310, 2049, 0), (320, 2176, 0),
                 (308, 4096, 0), (3, 4097, 0), (307, 4098, 0), (160, 5000, 0), (155, 6143, 0),
                 (156, 8192, 0), (153, 7001, 1), (153, 4104, 8),
                 (155, 6144, 0), (154, 6600, 0)]}


@pytest.mark.parametrize("dtype,rows,cols,extra", [(d, *s) for d in RINGS for s in RINGS[d]])
def test_backward_of_many_rows(dtype, rows, cols, extra):
    x, dy, up = (values(rows, cols, dtype, 130 + i, s) for i, s in enumerate((2.0, 0.1, 0.1)))
    gamma, n = vector(cols, 13), rng_of(cols)
    rstd = ref.norm(x, gamma, EPS)[1].float()
    layout = (0, extra)
    for dh, p in ((None, 0.0), (up, 0.0), (up, 0.2), (None, 0.3)):
        dx, dr = out(x, layout), out(x, layout)
        kw = dict(p=p, rng=n.cuda(), site=5, dresidual=dr.t) if p else {}
        got = fr.fr_rmsnorm_backward(put(dy, layout), put(x, layout), gamma.cuda(), rstd.cuda(), dx=dx.t,
                                     dh=None if dh is None else put(dh, layout), **kw)
        check_backward(x, gamma, dh, p, n, 5, got, dy, rstd, f"p {p} dh {dh is not None}")
        assert dx.intact() and (not p or dr.intact())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,extra", [(700, 255, 0), (700, 300, 1), (600, 511, 5), (2000, 200, 56),
                                             (500, 769, 2), (400, 2045, 3), (310, 4098, 6), (306, 8191, 0),
                                             (160, 16377, 0), (160, 16383, 4), (3000, 8, 0), (4100, 40, 0)])
def test_forward_of_many_rows(dtype, rows, cols, extra):
    """Rows in phase of every class, and the many short rows that lanes share."""
    x, r = values(rows, cols, dtype, 140), values(rows, cols, dtype, 141, 3.0)
    gamma, n = vector(cols, 14), rng_of(cols + 9)
    layout = (0, extra)
    for i, (res, p) in enumerate(((None, 0.0), (r, 0.0), (r, 0.2), (None, 0.5))):
        kw = {}
        y = out(x, layout)
        if p or res is not None:
            h = out(x, layout)
            kw = dict(h=h.t, p=p, rng=n.cuda(), site=6, residual=None if res is None else put(res, layout))
        got = fr.fr_rmsnorm(put(x, layout), gamma.cuda(), EPS, out=y.t, **kw)
        check_norm(x, res, p, n, 6, got, gamma, f"p {p} residual {res is not None}")
        assert y.intact() and (not kw or h.intact())
        q = out(x, layout, torch.float8_e4m3fn)
        scale = ("row", "group", torch.tensor([0.02]))[i % 3]
        s = scale if isinstance(scale, str) else "given"
        got = fr.fr_rmsnorm_quant(put(x, layout), gamma.cuda(), EPS, out=q.t,
                                  scale=scale if s != "given" else scale.cuda(), **kw)
        check_norm(x, res, p, n, 6, got, gamma, f"{s} p {p}", s, scale if s == "given" else None)
        assert q.intact()
        if p:
            d = out(x, layout)
            fr.fr_dropout(put(x, layout), p, n.cuda(), 6, out=d.t,
                          residual=None if res is None else put(res, layout))
            assert torch.equal(d.t, h.t) and d.intact()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(39011, 64), (19999, 128), (9737, 136), (9801, 256), (38920, 24),
                                       (16384, 128), (4865, 256)])
def test_more_short_rows_than_a_warp_takes_at_once(rows, cols, dtype):
    """The lanes of a warp share rows, several each; with every scale and with none."""
    x, r = values(rows, cols, dtype, 150), values(rows, cols, dtype, 151, 3.0)
    gamma, n = vector(cols, 15), rng_of(cols + 10)
    for res, p in ((None, 0.0), (r, 0.0), (r, 0.2)):
        kw = dict(p=p, rng=n.cuda(), site=7, residual=None if res is None else res.cuda())
        what = f"p {p} residual {res is not None}"
        got = fr.fr_rmsnorm(x.cuda(), gamma.cuda(), EPS, **kw)
        check_norm(x, res, p, n, 7, got, gamma, what)
        for quant in ("row", "group", "given"):
            given = torch.tensor([0.01])
            got = fr.fr_rmsnorm_quant(x.cuda(), gamma.cuda(), EPS, want_rstd=True,
                                      scale=given.cuda() if quant == "given" else quant, **kw)
            check_norm(x, res, p, n, 7, got, gamma, f"{what} {quant}", quant, given)


@pytest.mark.parametrize("rows,cols", [(7301, 2048), (6700, 2296), (1830, 8192), (1771, 8200), (920, 16384), (1400, 10512),
                                       (2950, 5120), (4200, 3584), (3300, 4608), (3250, 4600), (1100, 13824)])
def test_more_chunks_than_the_gpu_holds(rows, cols):
    """A warp takes eight chunks of a row (4 with a residual) when there are enough of them."""
    x, r = values(rows, cols, "bf16", 190), values(rows, cols, "bf16", 191, 3.0)
    gamma = vector(cols, 19)
    got = fr.fr_rmsnorm(x.cuda(), gamma.cuda(), EPS)
    check_norm(x, None, 0.0, None, 0, got, gamma, "norm")
    for i, quant in enumerate(("row", "group", "given")):
        given, res = torch.tensor([0.008]), r if i == rows % 3 else None
        got = fr.fr_rmsnorm_quant(x.cuda(), gamma.cuda(), EPS, want_rstd=True,
                                  scale=given.cuda() if quant == "given" else quant,
                                  residual=None if res is None else res.cuda())
        check_norm(x, res, 0.0, None, 0, got, gamma, quant, quant, given)


def test_neighbours_of_a_row_do_not_reach_it():
    """A unit at a row's edge holds elements of the rows beside it (or of the gap): whatever
    they are, the row's results are its own."""
    rows, cols, ld = 64, 1021, 1029
    x, dy = values(rows, cols, "bf16", 150), values(rows, cols, "bf16", 151)
    gamma, n = vector(cols, 15), rng_of(15)
    for bad in (math.nan, math.inf):
        def placed(v):
            buf = torch.full((rows, ld), bad, dtype=v.dtype, device="cuda")
            buf[1::2, :cols] = v[1::2].cuda()  # every other row is bad too
            return buf[:, :cols]

        odd = slice(1, None, 2)
        xb, dyb = placed(x), placed(dy)
        a = fr.fr_rmsnorm(xb, gamma.cuda(), EPS, residual=xb, p=0.3, rng=n.cuda())
        want = ref.dropout(x, 0.3, n, 0, x)
        ref.assert_near(a["h"][odd], want[odd], ref.dropout_bound(x, 0.3, x, want, x.dtype)[odd], "h")
        h = a["h"].cpu()[odd]
        y, rstd = ref.norm(h, gamma, EPS)
        ref.assert_near(a["rstd"][odd], rstd, ref.rstd_bound(cols) * rstd, "rstd")
        ref.assert_near(a["y"][odd], y, ref.norm_bound(cols, y, x.dtype), "y")
        rs = ref.norm(x, gamma, EPS)[1].float()
        b = fr.fr_rmsnorm_backward(dyb, xb, gamma.cuda(), rs.cuda(), dh=dyb)
        d, _ = ref.backward(dy, x, gamma, rs, dy)
        bound = ref.backward_bound(dy, x, gamma, rs, dy, d, x.dtype)
        ref.assert_near(b["dx"][odd], d[odd], bound[odd], "dx")


def test_more_rows_than_a_round_of_every_cta():
    """The row counts at which a CTA's rounds, row groups and pairs of rows end."""
    cols = 2048
    gamma = vector(cols, 16)
    for rows in (151, 152, 153, 303, 304, 305, 607, 608, 609, 1215, 1217):
        x, dy = values(rows, cols, "bf16", 160), values(rows, cols, "bf16", 161)
        rstd = ref.norm(x, gamma, EPS)[1].float()
        for p in (0.0, 0.1):
            n = rng_of(rows)
            got = fr.fr_rmsnorm_backward(dy.cuda(), x.cuda(), gamma.cuda(), rstd.cuda(), p=p, rng=n.cuda())
            check_backward(x, gamma, None, p, n, 0, got, dy, rstd, f"{rows} rows p {p}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,layout", [(20000, 64, (0, 0)), (12000, 63, (0, 0)), (6000, 500, (0, 4)),
                                              (6000, 505, (0, 0)), (10000, 7, (0, 2)), (6000, 300, (1, 0)),
                                              (700, 4096, (0, 0)), (650, 4101, (0, 0)), (600, 4100, (1, 1)),
                                              (310001, 1, (0, 0)), (160000, 9, (0, 0)), (76001, 20, (0, 4)),
                                              (40001, 63, (0, 0)), (20001, 121, (0, 5)), (2501, 987, (0, 2))])
def test_dropout_of_many_rows(rows, cols, layout, dtype):
    x, r = values(rows, cols, dtype, 170), values(rows, cols, dtype, 171)
    n = rng_of(cols + 17)
    for res in (None, r):
        o = out(x, layout)
        fr.fr_dropout(put(x, layout), 0.4, n.cuda(), 2, out=o.t,
                      residual=None if res is None else put(res, layout))
        want = ref.dropout(x, 0.4, n, 2, res)
        ref.assert_near(o.t, want, ref.dropout_bound(x, 0.4, res, want, DTYPES[dtype]))
        assert o.intact()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(5, 63), (9001, 505), (310001, 1), (33, 4097), (101, 17)])
def test_dropout_of_odd_rows_bit_for_bit(rows, cols, dtype):
    """Nothing dropped, everything dropped, in place, and out of phase: the same elements."""
    x, r = values(rows, cols, dtype, 180).cuda(), values(rows, cols, dtype, 181).cuda()
    n = rng_of(cols + 18).cuda()
    assert torch.equal(fr.fr_dropout(x, 0.0, None), x)
    assert torch.equal(fr.fr_dropout(x, 0.0, None, residual=r), (x.float() + r.float()).to(x.dtype))
    assert torch.equal(fr.fr_dropout(torch.full_like(x, float("nan")), 1.0, n, residual=r), r)
    want = fr.fr_dropout(x, 0.3, n, 2, residual=r)
    a, b = x.clone(), r.clone()
    assert torch.equal(fr.fr_dropout(a, 0.3, n, 2, residual=r, out=a), want)
    assert torch.equal(fr.fr_dropout(x, 0.3, n, 2, residual=b, out=b), want)
    v = torch.zeros(rows, cols + 9, device="cuda", dtype=x.dtype)[:, 1:1 + cols]
    v.copy_(x)
    assert torch.equal(fr.fr_dropout(v, 0.3, n, 2, residual=r), want)


@pytest.mark.parametrize("dtype,cols", [("bf16", 11008), ("bf16", 1000), ("bf16", 5120), ("f32", 5000), ("f32", 128)])
def test_gamma_at_any_address(dtype, cols):
    """A vector needs no more than its type's alignment; the gradient does not depend on it."""
    x, dy = values(310, cols, dtype, 200).cuda(), values(310, cols, dtype, 201, 0.1).cuda()
    gamma = vector(cols, 20).cuda()
    moved = torch.zeros(cols + 1, device="cuda")[1:]
    moved.copy_(gamma)
    rstd = fr.fr_rmsnorm(x, gamma, EPS)["rstd"]
    a, b = (fr.fr_rmsnorm_backward(dy, x, g, rstd) for g in (gamma, moved))
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dgamma"], b["dgamma"])


def test_auto_takes_a_form_that_holds_the_rows():
    """Long rows, aligned and not: the workspace that AUTO asks for serves either form."""
    for rows, cols in ((2, 8200), (3, 16384), (2, 16383), (1, 16392)):
        x, dy = values(rows, cols, "bf16", 180), values(rows, cols, "bf16", 181)
        gamma = vector(cols, 18)
        rstd = ref.norm(x, gamma, EPS)[1].float()
        for layout in LAYOUTS:
            got = fr.fr_rmsnorm(put(x, layout), gamma.cuda(), EPS)
            check_norm(x, None, 0.0, None, 0, got, gamma, f"{cols} {layout}")
            back = fr.fr_rmsnorm_backward(put(dy, layout), put(x, layout), gamma.cuda(), rstd.cuda())
            check_backward(x, gamma, None, 0.0, None, 0, back, dy, rstd, f"{cols} {layout}")


FIRST_CALLS = """
import sys; sys.path.insert(0, sys.argv[1])
import torch, reduction_pointwise_row_gb300 as fr
x = torch.randn(200, 4096, device="cuda").bfloat16(); r = torch.randn_like(x)
g = torch.ones(4096, device="cuda"); n = torch.tensor([3, 4], device="cuda")
fr.fr_workspace_size("rmsnorm_backward", 200, 4096, "bf16")
torch.cuda.synchronize()
def step():
    a = fr.fr_rmsnorm(x, g, residual=r, p=0.1, rng=n)
    b = fr.fr_rmsnorm_backward(x, a["h"], g, a["rstd"], dh=r, p=0.1, rng=n)
    q = fr.fr_rmsnorm_quant(x, g, scale="group")
    return [*a.values(), *b.values(), *q.values(), fr.fr_dropout(x, 0.2, n)]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    outs = step()
graph.replay(); torch.cuda.synchronize()
for o, e in zip(outs, step()):
    assert torch.equal(o.view(torch.uint8), e.view(torch.uint8))
print("same")
"""


def test_first_calls_within_a_capture():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS, root], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("cols,ld", [(1000, 1000), (1000, 1003), (1001, 1008), (1001, 1001), (64, 80), (7, 12)])
def test_outputs_share_the_phase_of_the_inputs(cols, ld):
    """New matrices lie as the inputs do within 8 elements; their values do not depend on it."""
    rows, n = 50, rng_of(6).cuda()
    x = values(rows, cols, "bf16", 190)
    v = put(x, (0, ld - cols))
    gamma = vector(cols, 19)
    a = fr.fr_rmsnorm(v, gamma.cuda(), EPS, residual=v, p=0.2, rng=n)
    q = fr.fr_rmsnorm_quant(v, gamma.cuda(), EPS)
    b = fr.fr_rmsnorm_backward(v, v, gamma.cuda(), a["rstd"], p=0.2, rng=n)
    for m in (a["y"], a["h"], q["y"], b["dx"], b["dresidual"], fr.fr_dropout(v, 0.2, n)):
        assert m.shape == (rows, cols) and (m.stride(0) - ld) % 8 == 0 and m.stride(0) < cols + 8
        assert m.is_contiguous() == ((ld - cols) % 8 == 0)
    check_norm(x, x, 0.2, n.cpu(), 0, a, gamma, "y")
    check_norm(x, None, 0.0, None, 0, q, gamma, "y8", "row")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [8, 150, 151, 154, 156, 500, 1001, 4097])
def test_the_workspace_holds_every_cta_s_share(cols, dtype):
    """Nothing is written past the bytes that fr_workspace_size gives, whatever the rows'
    number leaves of the classes of phases."""
    gamma, n = vector(cols, 21).cuda(), rng_of(21).cuda()
    for rows in [*range(1, 42), 151, 152, 153, 303, 305]:
        x, dy = values(rows, cols, dtype, 210).cuda(), values(rows, cols, dtype, 211).cuda()
        rstd = torch.ones(rows, device="cuda")
        nws = fr.fr_workspace_size("rmsnorm_backward", rows, cols, dtype)
        ws = torch.full((nws + 64 * 1024,), GUARD, dtype=torch.uint8, device="cuda")
        for p in (0.0, 0.5):
            fr.fr_rmsnorm_backward(dy, x, gamma, rstd, p=p, rng=n, workspace=ws[:nws])
            assert (ws[nws:] == GUARD).all(), rows


def test_vectors_end_where_they_end():
    """rstd, scales and dgamma are written to their last element and no further."""
    def guarded(shape):
        n = int(np.prod(shape))
        raw = torch.full((n + 64,), -7.0, device="cuda")
        return raw, raw[:n].view(shape)

    for dtype in DTYPES:
        for rows, cols in ((1, 1), (3, 129), (17, 128), (33, 1001), (300, 64), (5, 300), (9, 4097), (2, 17000)):
            x = values(rows, cols, dtype, 220)
            gamma = vector(cols, 22)
            groups = -(-cols // 128)
            for mode, shape in (("row", (rows,)), ("group", (rows, groups))):
                (r0, rstd), (s0, scale), (d0, dgamma) = (guarded(s) for s in ((rows,), shape, (cols,)))
                q = fr.fr_rmsnorm_quant(x.cuda(), gamma.cuda(), EPS, scale=mode, scale_out=scale, rstd=rstd)
                check_norm(x, None, 0.0, None, 0, q, gamma, f"{rows}x{cols} {mode}", mode)
                fr.fr_rmsnorm_backward(x.cuda(), x.cuda(), gamma.cuda(), rstd, dgamma=dgamma)
                want = ref.backward(x, x, gamma, rstd.cpu())[1]
                ref.assert_near(dgamma, want, ref.dgamma_bound(x, x, rstd.cpu()), "dgamma")
                for raw, v in ((r0, rstd), (s0, scale), (d0, dgamma)):
                    assert (raw[v.numel():] == -7.0).all()
