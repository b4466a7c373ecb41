"""The calls over rows of logits (fr_logprobs, fr_distill, fr_xent_backward and
the backward passes) against their 64-bit formulas: lengths, offsets and row
strides, masks, ties, special values, refusals on the device, streams and
graphs."""
import math

import numpy as np
import pytest
import torch

import logits_ref as ref
import reduction_pointwise_row_gb300 as fr

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# (rows, cols): one element to long rows, around vector, CTA and chunk sizes
SHAPES = [(1, 1), (3, 2), (2, 15), (4, 16), (5, 33), (7, 100), (3, 129), (33, 1000), (4, 1025),
          (3, 2048), (2, 4097), (3, 8191), (2, 16384), (300, 777), (2, 32001), (5, 50257),
          (1, 65537), (2, 131072), (1, 262145)]
# (first element's offset, elements added to the row stride)
LAYOUTS = [(0, 0), (1, 3), (5, 16), (8, 47)]


def rng(*key):
    return np.random.default_rng(list(key))


def placed(x, offset=0, extra=0, fill=float("nan")):
    """x on the GPU as a view into a larger buffer whose other elements are `fill`."""
    rows, cols = x.shape
    ld = cols + extra
    buf = torch.full((offset + rows * ld + 64,), fill, dtype=x.dtype, device="cuda")
    v = buf[offset:offset + rows * ld].as_strided((rows, cols), (ld, 1), offset)
    v.copy_(x)
    return buf, v


def untouched(buf, view, offset, extra):
    """Everything outside the view still holds NaN."""
    rows, cols = view.shape
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep.as_strided((rows, cols), (cols + extra, 1), offset).zero_()
    return bool(torch.isnan(buf[keep]).all())


def logits(rows, cols, dtype, seed, sigma=3.0):
    g = rng(seed, rows, cols)
    x = torch.from_numpy(g.normal(0.0, sigma, (rows, cols)).astype(np.float32))
    return x.to(DTYPES[dtype])


def tokens(rows, cols, seed, ignored=0.2):
    g = rng(seed, rows, cols, 7)
    t = torch.from_numpy(g.integers(0, cols, rows))
    t[torch.from_numpy(g.random(rows) < ignored)] = -100
    return t


def entries(rows, cols, top, seed, padding=0.3):
    g = rng(seed, rows, cols, top)
    i = torch.from_numpy(g.integers(0, cols, (rows, top)))  # repeats allowed
    i[torch.from_numpy(g.random((rows, top)) < padding)] = -1
    z = torch.from_numpy(g.normal(0.0, 3.0, (rows, top)).astype(np.float32))
    z[i < 0] = float("nan")  # a padding entry's logit is not looked at
    return i, z


def check_logprobs(x, got, t, top, what):
    """Each output in `got` against its formula."""
    cols = x.shape[1]
    r = ref.logprobs(x, t, top)
    e = ref.eps(cols)
    size = torch.nan_to_num(x.double().amax(1).abs(), posinf=0.0)
    bounds = {
        "logprob": lambda v: e + 4 * ref.U * torch.nan_to_num(v.abs(), posinf=0.0),
        "entropy": lambda v: e * (2 + 2 * math.log(cols)),
        "lse": lambda v: e + 2 * ref.U * (size + math.log(cols)),
        "top_logprob": lambda v: e + 4 * ref.U * torch.nan_to_num(v.abs(), posinf=0.0),
    }
    for k, o in got.items():
        if k == "top_index":
            assert torch.equal(o.cpu(), r[k]), f"{what} top_index"
        else:
            ref.assert_near(o, r[k], bounds[k](r[k]), f"{what} {k}")


def forms(*names):
    return pytest.mark.parametrize("form", names)


def skip_long(form, cols, dtype):
    if form == "persistent" and cols * (2 if dtype == "bf16" else 4) >= 129 * 32:
        pytest.skip("a row longer than a warp's registers")


FORWARD_FORMS = forms("looped", "split", "persistent")
BACKWARD_FORMS = forms("looped", "persistent", "split")


@FORWARD_FORMS
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_logprobs_shapes(rows, cols, dtype, form):
    skip_long(form, cols, dtype)
    for n, (offset, extra) in enumerate(LAYOUTS):
        x = logits(rows, cols, dtype, 11 + n)
        t = tokens(rows, cols, n)
        _, v = placed(x, offset, extra, fill=math.inf)
        for top in sorted({0, 1, min(5, cols), min(20, cols), min(64, cols), min(128, cols)}):
            got = fr.fr_logprobs(v, t.cuda(), top=top, form=form)
            check_logprobs(x, got, t, top, f"{rows}x{cols} {dtype} {offset},{extra} top {top}")
    assert fr.fr_check_device_error() == 0


def special_rows(cols, dtype):
    """Rows that a mask, a tie or a special value makes hard, by name."""
    lowest = torch.finfo(DTYPES[dtype]).min
    g = rng(cols, 3)
    base = torch.from_numpy(g.normal(0.0, 3.0, cols).astype(np.float32))
    ramp = torch.linspace(-20.0, 20.0, cols)
    some = torch.from_numpy(g.permutation(cols)[:max(1, min(3, cols))])

    def few(fill):
        r = torch.full((cols,), fill)
        r[some] = torch.tensor([1.0, 2.0, -3.0])[:len(some)]
        return r

    def put(value, at=None):
        r = base.clone()
        r[cols // 2 if at is None else at] = value
        return r

    zeros = torch.zeros(cols)
    zeros[::2] = -0.0
    clustered = base.clone()
    clustered[:min(cols, 700)] += 100.0  # the largest all in a few chunks
    rows = {
        "all -inf": torch.full((cols,), -math.inf), "all lowest": torch.full((cols,), lowest),
        "few, -inf": few(-math.inf), "few, lowest": few(lowest), "constant": torch.full((cols,), 2.5),
        "zeros of both signs": zeros, "rising": ramp, "falling": ramp.flip(0),
        "two values": (torch.arange(cols) % 2).float(), "clustered": clustered,
        "a NaN": put(math.nan), "NaN first and last": put(math.nan, torch.tensor([0, cols - 1])),
        "+inf": put(math.inf), "-inf here and there": put(-math.inf, slice(0, None, 3)),
        "one far above": put(200.0), "large offset": base + 30000.0,
        "all large": torch.full((cols,), 1e30), "all NaN": torch.full((cols,), math.nan),
        "lowest and -inf": torch.where(torch.arange(cols) % 2 == 0, lowest, -math.inf),
    }
    return list(rows), torch.stack(list(rows.values())).to(DTYPES[dtype])


@FORWARD_FORMS
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [1, 2, 40, 129, 1000, 1500, 5000, 33000, 50257])
def test_logprobs_special_rows(cols, dtype, form):
    skip_long(form, cols, dtype)
    names, x = special_rows(cols, dtype)
    t = torch.from_numpy(rng(cols).integers(0, cols, len(names)))
    v = x.cuda()
    for top in sorted({1, min(20, cols), min(128, cols)}):
        got = fr.fr_logprobs(v, t.cuda(), top=top, form=form)
        for i, name in enumerate(names):
            one = {k: o[i:i + 1] for k, o in got.items()}
            check_logprobs(x[i:i + 1], one, t[i:i + 1], top, f"{name} of {cols} {dtype} top {top}")
    assert fr.fr_check_device_error() == 0


@FORWARD_FORMS
def test_logprobs_outputs_are_optional(form):
    x = logits(9, 2000, "bf16", 5)  # short enough for every form
    v, t = x.cuda(), tokens(9, 2000, 5)
    only = [dict(token=t.cuda(), want_entropy=False, want_lse=False), dict(want_lse=False),
            dict(want_entropy=False), dict(want_entropy=False, want_lse=False, top=7)]
    names = [["logprob"], ["entropy"], ["lse"], ["top_index", "top_logprob"]]
    for kw, name in zip(only, names):
        got = fr.fr_logprobs(v, form=form, **kw)
        assert sorted(got) == name
        check_logprobs(x, got, t, kw.get("top", 0), str(name))
    assert sorted(fr.fr_logprobs(v, top=3)) == ["entropy", "lse", "top_index", "top_logprob"]


@forms("auto", "looped")
def test_bad_tokens_and_indexes_are_recorded(form):
    x = logits(6, 500, "bf16", 8).cuda()
    t = torch.tensor([0, 500, -1, 499, -100, 1 << 40])
    got = fr.fr_logprobs(x, t.cuda(), form=form)["logprob"].cpu()
    assert torch.isnan(got).tolist() == [False, True, True, False, False, True]
    assert got[4] == 0
    assert fr.fr_check_device_error() == 1
    assert fr.fr_check_device_error() == 0
    d = fr.fr_logprobs_backward(x, t.cuda(), dlogprob=torch.ones(6, device="cuda"), form=form)
    assert torch.isnan(d).all(1).tolist() == [False, True, True, False, False, True]
    assert (d[4] == 0).all()
    assert fr.fr_check_device_error() == 1
    r = fr.fr_xent_backward(x, t.cuda(), torch.ones(1, device="cuda"), form=form)
    assert torch.isnan(r["dlogits"]).all(1).tolist() == [False, True, True, False, False, True]
    assert torch.isnan(r["loss"]).tolist() == [False, True, True, False, False, True]
    assert fr.fr_check_device_error() == 1
    i = torch.tensor([[0, 1], [500, 1], [1, 1 << 40], [-1, -5], [3, 3], [-1, 2]])
    z = torch.ones(6, 2)
    loss = fr.fr_distill(x, i.cuda(), z.cuda(), form=form)
    assert torch.isnan(loss).tolist() == [False, True, True, False, False, False]
    assert loss[3] == 0
    assert fr.fr_check_device_error() == 1
    r = fr.fr_distill_backward(x, i.cuda(), z.cuda(), torch.ones(6, device="cuda"), form=form)
    assert torch.isnan(r["dlogits"]).all(1).tolist() == [False, True, True, False, False, False]
    assert torch.isnan(r["loss"]).tolist() == [False, True, True, False, False, False]
    assert (r["dlogits"][3] == 0).all()
    assert fr.fr_check_device_error() == 1


def loss_bound(x, r, index, logit, temperature):
    """T^2 sum q (log q - log p): each log within EPS plus its own rounding."""
    _, _, logp, _ = ref.parts(x, temperature)
    q, logq, _ = ref.teacher(index, logit, temperature)
    at = logp.gather(1, index.clamp(0, x.shape[1] - 1))
    size = torch.nan_to_num(q * (logq.abs() + at.abs() + 1), nan=0.0, posinf=0.0).sum(1)
    return temperature ** 2 * size * (2 * ref.eps(x.shape[1]) + 160 * ref.U)


@FORWARD_FORMS
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_distill_shapes(rows, cols, dtype, form):
    skip_long(form, cols, dtype)
    for n, ((offset, extra), top) in enumerate(zip(LAYOUTS, (1, 20, 65, 128))):
        temperature = (1.0, 2.0, 0.7, 4.0)[n]
        x = logits(rows, cols, dtype, 31 + n)
        i, z = entries(rows, cols, top, n)
        _, v = placed(x, offset, extra, fill=math.inf)
        got = fr.fr_distill(v, i.cuda(), z.cuda(), temperature, form=form)
        r = ref.distill(x, i, z, temperature)
        ref.assert_near(got, r, loss_bound(x, r, i, z, temperature),
                        f"{rows}x{cols} {dtype} top {top}")
    assert fr.fr_check_device_error() == 0


# ---- gradients ------------------------------------------------------------------

def out_of_phase(x, n):
    """Layouts of dlogits: the logits' own phase, another one, in place."""
    return [(0, 0), (3, 5), None][n % 3]


def run_backward(op, x, layout, dlayout, form, **kw):
    """(gradient, loss or None) of the call on a copy of x at `layout`, the
    gradient written at `dlayout` (None: over the logits)."""
    if form == "persistent" and x.shape[1] * x.element_size() > 200000:
        pytest.skip("a row longer than shared memory")
    buf, v = placed(x, *layout)
    if dlayout is None:
        dbuf, out, dlayout = buf, v, layout
    else:
        dbuf, out = placed(torch.full_like(x, 77.0), *dlayout)
    got = op(v, dlogits=out, form=form, **kw)
    d, loss = (got["dlogits"], got.get("loss")) if isinstance(got, dict) else (got, None)
    assert d.data_ptr() == out.data_ptr()
    assert untouched(dbuf, out, *dlayout), "written outside the rows"
    return out.clone(), loss


def upstream(rows, seed, one=False):
    return torch.from_numpy(rng(rows, seed, 5).normal(0.0, 1.0, 1 if one else rows)
                            .astype(np.float32))


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


@BACKWARD_FORMS
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_logprobs_backward_shapes(rows, cols, dtype, form):
    for n, layout in enumerate(LAYOUTS):
        x = logits(rows, cols, dtype, 51 + n)
        t = tokens(rows, cols, n)
        g, h = upstream(rows, n, one=n == 1), upstream(rows, n + 9, one=n == 2)
        for use in ((g, h), (g, None), (None, h)):
            d, _ = run_backward(fr.fr_logprobs_backward, x, layout, out_of_phase(x, n), form,
                                token=t.cuda() if use[0] is not None else None,
                                dlogprob=cuda(use[0])[0], dentropy=cuda(use[1])[0])
            r = ref.logprobs_backward(x, t, use[0], use[1])
            b = ref.gradient_bound(x, r, torch.zeros(1) if use[0] is None else use[0], use[1])
            ref.assert_near(d, r, b, f"{rows}x{cols} {dtype} {n}")


@BACKWARD_FORMS
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_xent_backward_shapes(rows, cols, dtype, form):
    for n, layout in enumerate(LAYOUTS):
        x = logits(rows, cols, dtype, 71 + n)
        t = tokens(rows, cols, n + 3)
        g = upstream(rows, n, one=n % 2 == 1)
        d, loss = run_backward(fr.fr_xent_backward, x, layout, out_of_phase(x, n + 1), form,
                               target=t.cuda(), dloss=g.cuda())
        r = ref.xent_backward(x, t, g)
        ref.assert_near(d, r, ref.gradient_bound(x, r, g), f"{rows}x{cols} {dtype} {n}")
        rl = ref.xent(x, t)
        ref.assert_near(loss, rl, ref.eps(cols) + 4 * ref.U * rl.abs(), "loss")


@BACKWARD_FORMS
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_distill_backward_shapes(rows, cols, dtype, form):
    for n, (layout, top) in enumerate(zip(LAYOUTS, (128, 1, 20, 65))):
        temperature = (2.0, 1.0, 4.0, 0.7)[n]
        x = logits(rows, cols, dtype, 91 + n)
        i, z = entries(rows, cols, top, n + 3)
        g = upstream(rows, n, one=n % 2 == 0)
        d, loss = run_backward(fr.fr_distill_backward, x, layout, out_of_phase(x, n + 2), form,
                               teacher_index=i.cuda(), teacher_logit=z.cuda(), dloss=g.cuda(),
                               temperature=temperature)
        r = ref.distill_backward(x, i, z, g, temperature)
        b = ref.gradient_bound(x, r, g * temperature, temperature=temperature)
        # the entries' weights, each within 64 u of its share, add up at the size of g T
        q, _, _ = ref.teacher(i, z, temperature)
        dense = torch.zeros_like(r).scatter_add_(1, i.clamp(min=0), q)
        b = b + (g.double().abs().expand(rows)[:, None] * temperature) * dense * 160 * ref.U
        ref.assert_near(d, r, b, f"{rows}x{cols} {dtype} {n}")
        rl = ref.distill(x, i, z, temperature)
        ref.assert_near(loss, rl, loss_bound(x, rl, i, z, temperature), "loss")


@BACKWARD_FORMS
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [1, 2, 40, 1000, 5000, 50257])
def test_gradients_of_special_rows(cols, dtype, form):
    names, x = special_rows(cols, dtype)
    rows = len(names)
    t = torch.from_numpy(rng(cols, 1).integers(0, cols, rows))
    g, h = upstream(rows, 1), upstream(rows, 2)
    i, z = entries(rows, cols, 9, 4, padding=0.1)
    for inplace in (False, True):
        lay = None if inplace else (0, 0)
        d, _ = run_backward(fr.fr_logprobs_backward, x, (0, 0), lay, form, token=t.cuda(),
                            dlogprob=g.cuda(), dentropy=h.cuda())
        r = ref.logprobs_backward(x, t, g, h)
        b = ref.gradient_bound(x, r, g, h)
        e, loss = run_backward(fr.fr_xent_backward, x, (0, 0), lay, form, target=t.cuda(),
                               dloss=g.cuda())
        re = ref.xent_backward(x, t, g)
        be = ref.gradient_bound(x, re, g)
        k, kl = run_backward(fr.fr_distill_backward, x, (0, 0), lay, form, teacher_index=i.cuda(),
                             teacher_logit=z.cuda(), dloss=g.cuda())
        rk = ref.distill_backward(x, i, z, g)
        bk = ref.gradient_bound(x, rk, g) + g.double().abs()[:, None] * 160 * ref.U
        rl, rkl = ref.xent(x, t), ref.distill(x, i, z)
        for n, name in enumerate(names):
            s = slice(n, n + 1)
            ref.assert_near(d[s], r[s], b[s], f"{name}: logprobs of {cols} {dtype}")
            ref.assert_near(e[s], re[s], be[s], f"{name}: xent of {cols} {dtype}")
            ref.assert_near(k[s], rk[s], bk[s], f"{name}: distill of {cols} {dtype}")
            ref.assert_near(loss[s], rl[s], ref.eps(cols) + 4 * ref.U * torch.nan_to_num(
                rl[s].abs(), posinf=0.0), f"{name}: loss")
            ref.assert_near(kl[s], rkl[s], loss_bound(x, rkl, i, z, 1.0)[s], f"{name}: kl")


@BACKWARD_FORMS
def test_teacher_rows(form):
    """Rows without weight, entries of -inf, the same index twice, one entry, a row
    stride past the entries."""
    cols = 3000
    fwd = "looped" if form == "looped" else "split"
    ninf = -math.inf
    i = torch.tensor([[-1, -1, -1, -1], [5, 6, 7, 8], [5, 6, 7, 8], [9, 9, 9, 9], [-1, -1, 4, -1],
                      [2999, 0, 2999, 0]])
    z = torch.tensor([[1.0, 2, 3, 4], [ninf] * 4, [1.0, ninf, 2.0, ninf], [0.5, 1.0, 2.0, -1.0],
                      [math.nan, math.nan, -3.0, ninf], [80.0, 79.0, -90.0, 0.0]])
    x = logits(6, cols, "f32", 2)
    g = upstream(6, 3)
    wide_i = torch.full((6, 11), 1 << 50)
    wide_z = torch.full((6, 11), math.nan)
    wide_i[:, :4], wide_z[:, :4] = i, z
    vi, vz = wide_i.cuda()[:, :4], wide_z.cuda()[:, :4]
    r = fr.fr_distill_backward(x.cuda(), vi, vz, g.cuda(), 2.0, form=form)
    rd, rl = ref.distill_backward(x, i, z, g, 2.0), ref.distill(x, i, z, 2.0)
    ref.assert_near(r["dlogits"], rd, ref.gradient_bound(x, rd, 2 * g, temperature=2.0)
                    + g.double().abs()[:, None] * 320 * ref.U, "dlogits")
    ref.assert_near(r["loss"], rl, loss_bound(x, rl, i, z, 2.0), "loss")
    ref.assert_near(fr.fr_distill(x.cuda(), vi, vz, 2.0, form=fwd), rl,
                    loss_bound(x, rl, i, z, 2.0), "loss alone")
    assert (r["dlogits"][:2] == 0).all() and (r["loss"][:2] == 0).all()
    # a weighted entry at a masked logit: +inf; an entry without weight there: nothing
    x[:, 6] = ninf
    loss = fr.fr_distill(x.cuda(), vi, vz, 2.0, form=fwd)
    assert torch.isfinite(loss).all()
    z[1] = torch.tensor([0.0, 0.0, 0.0, 0.0])
    assert fr.fr_distill(x.cuda(), i.cuda(), z.cuda(), 2.0, form=fwd)[1] == math.inf
    assert fr.fr_check_device_error() == 0


@BACKWARD_FORMS
def test_gradients_against_differences(form):
    """Central differences of the 64-bit formulas, step 2^-10: their error is
    step^2 / 6 times a third derivative of at most 8 (per unit of upstream)."""
    rows, cols, step = 4, 700, 2.0 ** -10
    x = logits(rows, cols, "f32", 6)
    t = torch.from_numpy(rng(1).integers(0, cols, rows))
    i, z = entries(rows, cols, 12, 1, padding=0.2)
    one = torch.ones(1, device="cuda")
    probe = torch.from_numpy(rng(2).integers(0, cols, 24)).tolist() + t.tolist() + \
        i[i >= 0].tolist()[:24]
    v = x.cuda()
    calls = [
        (lambda y: ref.logprobs(y, t)["logprob"],
         fr.fr_logprobs_backward(v, t.cuda(), dlogprob=one, form=form)),
        (lambda y: ref.logprobs(y)["entropy"], fr.fr_logprobs_backward(v, dentropy=one, form=form)),
        (lambda y: ref.distill(y, i, z, 2.0),
         fr.fr_distill_backward(v, i.cuda(), z.cuda(), one, 2.0, form=form)["dlogits"]),
        (lambda y: ref.xent(y, t), fr.fr_xent_backward(v, t.cuda(), one, form=form)["dlogits"]),
    ]
    for f, d in calls:
        for j in probe:
            up, down = x.double(), x.double()
            up[:, j] += step
            down[:, j] -= step
            slope = (f(up) - f(down)) / (2 * step)
            ref.assert_near(d[:, j], slope, 4 * (8 * step ** 2 / 6 + 16 * ref.eps(cols)), f"at {j}")


# ---- together, and with what was there ---------------------------------------------

def test_a_teacher_scores_and_a_student_learns():
    """A teacher's alternatives go into the student's step as they are; training
    against fr_xent agrees with fr_xent's own results."""
    rows, cols, top = 40, 50257, 32
    tx, sx = logits(rows, cols, "bf16", 1), logits(rows, cols, "bf16", 2)
    t = tokens(rows, cols, 4)
    scored = fr.fr_logprobs(tx.cuda(), t.cuda(), top=top)
    v = sx.cuda()
    step = fr.fr_distill_backward(v, scored["top_index"], scored["top_logprob"],
                                  torch.full((1,), 1.0 / rows, device="cuda"), 2.0)
    i, z = scored["top_index"].cpu(), tx.float().gather(1, scored["top_index"].cpu())
    g = torch.full((1,), 1.0 / rows)
    rl, rd = ref.distill(sx, i, z, 2.0), ref.distill_backward(sx, i, z, g, 2.0)
    # the teacher's log probabilities carry EPS each
    ref.assert_near(step["loss"], rl, loss_bound(sx, rl, i, z, 2.0) + 60 * ref.eps(cols), "loss")
    ref.assert_near(step["dlogits"], rd, ref.gradient_bound(sx, rd, 2 * g, temperature=2.0)
                    + 4 * ref.eps(cols) / rows, "dlogits")
    # the forward call sums in another order: each is within its bound of the formula
    ref.assert_near(fr.fr_distill(v, scored["top_index"], scored["top_logprob"], 2.0), rl,
                    loss_bound(sx, rl, i, z, 2.0) + 60 * ref.eps(cols), "loss alone")
    # beside fr_xent: its loss, its argmax and its gradient
    x1 = fr.fr_xent(v, t.cuda(), -100, want_argmax=True)
    x2 = fr.fr_xent_backward(v, t.cuda(), torch.ones(1, device="cuda"))
    lp = fr.fr_logprobs(v, t.cuda(), top=1)
    bound = 2 * ref.eps(cols) + 16 * ref.U * 20
    ref.assert_near(x2["loss"], x1["loss"].cpu(), bound, "xent")
    ref.assert_near(-lp["logprob"], x1["loss"].cpu(), bound, "logprob")
    assert torch.equal(lp["top_index"][:, 0], x1["argmax"])
    d = fr.fr_logprobs_backward(v, t.cuda(), dlogprob=-torch.ones(1, device="cuda"))
    assert torch.equal(d, x2["dlogits"])


def step_of_all(x, t, i, z, g, scratch):
    """All five calls as one sequence; the last gradient overwrites its logits."""
    a = fr.fr_logprobs(x, t, top=11)
    b = fr.fr_distill(x, i, z, 1.5)
    c = fr.fr_distill_backward(x, i, z, g, 1.5)
    d = fr.fr_logprobs_backward(x, t, dlogprob=g, dentropy=a["entropy"])
    scratch.copy_(x)
    e = fr.fr_xent_backward(scratch, t, g, dlogits=scratch)
    return [*a.values(), b, c["loss"], c["dlogits"], d, e["loss"], e["dlogits"]]


@pytest.mark.parametrize("rows,cols", [(1, 50257), (37, 50257), (700, 4097)])
def test_captured_replayed_and_on_other_streams(rows, cols):
    """A captured graph's replay on new data, two graphs replayed at once on two
    streams, and a call on a side stream give what eager calls give."""
    def data(seed):
        x = logits(rows, cols, "bf16", seed).cuda()
        i, z = (v.cuda() for v in entries(rows, cols, 17, seed))
        return [x, tokens(rows, cols, seed).cuda(), i, z, upstream(rows, seed).cuda()]

    def eager(inputs):
        out = [o.clone() for o in step_of_all(*inputs, torch.empty_like(inputs[0]))]
        torch.cuda.synchronize()
        return out

    graphs = []
    for seed in (1, 2):
        held = [v.clone() for v in data(seed)]
        scratch = torch.empty_like(held[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step_of_all(*held, scratch)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step_of_all(*held, scratch)
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
    for (_, held, outs) in graphs:
        for o, e in zip(outs, eager(held)):
            assert torch.equal(o.nan_to_num(7.0), e.nan_to_num(7.0))
    # the stream argument: inputs made on the current stream, the call on another
    x, t, i, z, g = data(9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fr.fr_distill_backward(x, i, z, g, 1.5, stream=s)
    lp = fr.fr_logprobs(x, t, top=4, stream=s)
    s.synchronize()
    want = fr.fr_distill_backward(x, i, z, g, 1.5)
    assert torch.equal(got["dlogits"], want["dlogits"])
    assert torch.equal(lp["top_index"], fr.fr_logprobs(x, t, top=4)["top_index"])


@pytest.mark.parametrize("rows,cols", [(5, 50257), (400, 1000)])
def test_runs_repeat_bit_for_bit(rows, cols):
    x = logits(rows, cols, "bf16", 3).cuda()
    i, z = (v.cuda() for v in entries(rows, cols, 30, 3))
    t, g = tokens(rows, cols, 3).cuda(), upstream(rows, 3).cuda()
    scratch = torch.empty_like(x)
    first = [o.clone() for o in step_of_all(x, t, i, z, g, scratch)]
    for _ in range(5):
        for o, f in zip(step_of_all(x, t, i, z, g, scratch), first):
            assert torch.equal(o.nan_to_num(7.0), f.nan_to_num(7.0))


def test_row_offsets_past_32_bits():
    """Rows whose elements lie past 2^32 bytes and 2^31 elements of their base."""
    cols, ld = 5001, (1 << 31) + 24
    buf = torch.empty(2 * ld + 2 * cols, dtype=torch.bfloat16, device="cuda")
    v = buf.as_strided((3, cols), (ld, 1), 0)
    x = logits(3, cols, "bf16", 1)
    v.copy_(x)
    t, g = tokens(3, cols, 1, ignored=0.0), upstream(3, 1)
    check_logprobs(x, fr.fr_logprobs(v, t.cuda(), top=9), t, 9, "far rows")
    i, z = entries(3, cols, 5, 1)
    r = ref.distill_backward(x, i, z, g)
    d = fr.fr_distill_backward(v, i.cuda(), z.cuda(), g.cuda(), dlogits=v)["dlogits"]
    ref.assert_near(d, r, ref.gradient_bound(x, r, g) + g.double().abs()[:, None] * 160 * ref.U)


def test_the_binding_refuses():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    g = torch.ones(4, device="cuda")
    i, z = torch.zeros(4, 3, dtype=torch.int64, device="cuda"), torch.zeros(4, 3, device="cuda")
    bad = [
        lambda: fr.fr_logprobs(x.half(), t), lambda: fr.fr_logprobs(x[:, ::2], t),
        lambda: fr.fr_logprobs(x.t(), t), lambda: fr.fr_logprobs(x[0], t),
        lambda: fr.fr_logprobs(x[:0], t[:0]), lambda: fr.fr_logprobs(x[:1].expand(4, 64), t),
        lambda: fr.fr_logprobs(x, t.int()), lambda: fr.fr_logprobs(x, t[:3]),
        lambda: fr.fr_logprobs(x, t[:2].repeat_interleave(4)[::2]),
        lambda: fr.fr_logprobs(x, t, top=65), lambda: fr.fr_logprobs(x, t, top=-1),
        lambda: fr.fr_logprobs(x, t.cpu()),
        lambda: fr.fr_logprobs(x, None, want_entropy=False, want_lse=False),
        lambda: fr.fr_logprobs_backward(x, t), lambda: fr.fr_logprobs_backward(x, None, g),
        lambda: fr.fr_logprobs_backward(x, t, g.double()),
        lambda: fr.fr_logprobs_backward(x, t, g[:3]),
        lambda: fr.fr_logprobs_backward(x, t, g, dlogits=x.float()),
        lambda: fr.fr_logprobs_backward(x, t, g, dlogits=x[:, :32]),
        lambda: fr.fr_distill(x, i, z[:, :2]), lambda: fr.fr_distill(x, i.int(), z),
        lambda: fr.fr_distill(x, i, z.bfloat16()), lambda: fr.fr_distill(x, i[:, :0], z[:, :0]),
        lambda: fr.fr_distill(x, i.expand(4, 3)[:, [0] * 129], z[:, [0] * 129]),
        lambda: fr.fr_distill(x, i[:1].expand(4, 3), z[:1].expand(4, 3)),
        lambda: fr.fr_distill_backward(x, i, z, g.cpu()),
        lambda: fr.fr_xent_backward(x, t, torch.ones(4, 1, device="cuda")),
    ]
    for n, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("accepted", n)
    for temperature in (0.0, -1.0, math.inf, math.nan, 1e-39):
        with pytest.raises(fr.FRError):
            fr.fr_distill(x, i, z, temperature)
    with pytest.raises(fr.FRError):  # in place over another row stride
        fr.fr_xent_backward(x[:2, :32], t[:2], g[:2], dlogits=x.view(-1).as_strided((2, 32), (32, 1)))
    with pytest.raises(fr.FRError):  # longer than a warp's registers, than shared memory
        fr.fr_logprobs(torch.zeros(1, 5000, device="cuda"), form="persistent")
    with pytest.raises(fr.FRError):
        fr.fr_xent_backward(torch.zeros(4, 70000, device="cuda"), t, g, form="persistent")


def test_upstream_gradients_with_a_stride():
    x, t = logits(50, 300, "f32", 4), tokens(50, 300, 4)
    pairs = upstream(100, 4).view(50, 2)
    g = pairs.cuda()[:, 1]
    assert g.stride(0) == 2
    got = fr.fr_xent_backward(x.cuda(), t.cuda(), g)
    want = fr.fr_xent_backward(x.cuda(), t.cuda(), g.contiguous())
    assert torch.equal(got["dlogits"], want["dlogits"])
    one = torch.full((), 0.25, device="cuda")
    got = fr.fr_xent_backward(x.cuda(), t.cuda(), one.expand(50), want_loss=False)
    assert list(got) == ["dlogits"]
    want = fr.fr_xent_backward(x.cuda(), t.cuda(), torch.full((50,), 0.25, device="cuda"))
    assert torch.equal(got["dlogits"], want["dlogits"])


def test_gradients_of_a_view_keep_its_phase():
    """A new dlogits for rows of a padded matrix shares their offset within 32 bytes,
    and a far row stride is not copied."""
    wide = logits(6, 1088, "bf16", 1).cuda()
    x, t = wide[:, :1001], tokens(6, 1001, 1).cuda()
    d = fr.fr_xent_backward(x, t, torch.ones(1, device="cuda"))["dlogits"]
    assert d.shape == x.shape and (d.stride(0) - x.stride(0)) % 16 == 0 and d.stride(0) < 1017
    far = wide.view(2, 3, 1088)[:, -1, :1001]
    d = fr.fr_xent_backward(far, t[:2], torch.ones(1, device="cuda"))["dlogits"]
    assert d.stride(0) < 1017


def test_a_workspace_of_the_callers_own():
    """The looped form's alternatives in a workspace of the caller's: used again, too
    small, misaligned, and not needed where another form runs."""
    rows, cols = 700, 4099
    x, t = logits(rows, cols, "bf16", 1), tokens(rows, cols, 1)
    v, tc = x.cuda(), t.cuda()
    n = fr.fr_workspace_size("logprobs", rows, cols, "bf16")
    assert n > 0 and fr.fr_auto_form("logprobs", rows, cols, "bf16", fr.sm_count()) == "looped"
    ws = torch.empty(n + 16, dtype=torch.uint8, device="cuda")
    for seed in (1, 2):
        x = logits(rows, cols, "bf16", seed)
        v.copy_(x)
        check_logprobs(x, fr.fr_logprobs(v, tc, top=9, workspace=ws), t, 9, f"seed {seed}")
    for bad in (ws[:n - 1], ws[8:n + 8]):
        with pytest.raises(fr.FRError):
            fr.fr_logprobs(v, tc, top=9, workspace=bad)
    assert fr.fr_workspace_size("logprobs", 5, cols, "bf16") == 0
    check_logprobs(x[:5], fr.fr_logprobs(v[:5], tc[:5], top=9), t[:5], 9, "few rows")


def test_calls_on_two_streams_at_once():
    """Eager calls of every kind interleaved on two streams, each with its own data."""
    data = []
    for seed in (1, 2):
        rows, cols = 650 + seed, 9001
        x = logits(rows, cols, "bf16", seed)
        i, z = entries(rows, cols, 30, seed)
        data.append((x, tokens(rows, cols, seed), i, z, upstream(rows, seed)))
    held = [[v.cuda() for v in d] for d in data]
    scratch = [torch.empty_like(h[0]) for h in held]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [None, None]
    for _ in range(4):
        for n, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[n] = step_of_all(*held[n], scratch[n])
    torch.cuda.synchronize()
    for n in range(2):
        for o, e in zip(outs[n], step_of_all(*held[n], scratch[n])):
            assert torch.equal(o.nan_to_num(7.0), e.nan_to_num(7.0))
    assert fr.fr_check_device_error() == 0


@pytest.mark.parametrize("rows", [1, 150, 153, 457, 1200])
def test_row_counts_around_the_device(rows):
    """Fewer rows than SMs, a few more, several a CTA: every row is written once, by
    the staged form whose CTAs take rows from one another and by the rule's choice."""
    cols = 9000
    x, t, g = logits(rows, cols, "bf16", 3), tokens(rows, cols, 3), upstream(rows, 3)
    r = ref.xent_backward(x, t, g)
    b = ref.gradient_bound(x, r, g)
    for form in ("persistent", "split", "auto"):
        for _ in range(3):
            d, _ = run_backward(fr.fr_xent_backward, x, (0, 0), (0, 0), form, target=t.cuda(),
                                dloss=g.cuda())
            ref.assert_near(d, r, b, f"{rows} rows {form}")


def test_all_rows_ignored_and_all_rows_bad():
    x = logits(400, 12000, "f32", 2).cuda()
    g = torch.ones(1, device="cuda")
    for form in ("looped", "persistent", "split"):
        r = fr.fr_xent_backward(x, torch.full((400,), -100, device="cuda"), g, form=form)
        assert (r["dlogits"] == 0).all() and (r["loss"] == 0).all()
        assert fr.fr_check_device_error() == 0
        r = fr.fr_xent_backward(x, torch.full((400,), 12000, device="cuda"), g, form=form)
        assert torch.isnan(r["dlogits"]).all() and torch.isnan(r["loss"]).all()
        assert fr.fr_check_device_error() == 1


@pytest.mark.parametrize("cols", [600, 20000, 90001])
def test_teacher_entries_that_repeat(cols):
    """The same index in many entries, in different lanes and registers; indexes that
    share a hash; all entries at one element."""
    top, rows = 128, 5
    i = torch.arange(top).repeat(rows, 1) * (cols // top)
    i[1, ::2] = i[1, 1]
    i[2, 64:] = i[2, :64]
    i[3] = 7
    i[4] = (torch.arange(top) % 2) * 256 + 3  # two indexes of one hash, 64 times each
    x, g = logits(rows, cols, "f32", 8), upstream(rows, 8)
    z = torch.from_numpy(rng(8, cols).normal(0, 2, (rows, top)).astype(np.float32))
    r = ref.distill_backward(x, i, z, g)
    q, _, _ = ref.teacher(i, z, 1.0)
    dense = torch.zeros_like(r).scatter_add_(1, i, q)
    b = ref.gradient_bound(x, r, g) + g.double().abs()[:, None] * dense * 320 * ref.U
    for form in ("looped", "split", "auto"):
        d, _ = run_backward(fr.fr_distill_backward, x, (0, 0), (0, 0), form,
                            teacher_index=i.cuda(), teacher_logit=z.cuda(), dloss=g.cuda())
        ref.assert_near(d, r, b, f"{cols} {form}")


def test_upstream_gradients_that_are_not_finite():
    """An infinite or NaN upstream gradient reaches its own row alone."""
    x, t = logits(4, 9000, "f32", 4), torch.tensor([0, 5, 7, -100])
    g = torch.tensor([1.0, math.inf, math.nan, math.inf])
    for form in ("looped", "persistent", "split"):
        d = fr.fr_xent_backward(x.cuda(), t.cuda(), g.cuda(), form=form)["dlogits"].cpu()
        r = ref.xent_backward(x[:1], t[:1], g[:1])
        ref.assert_near(d[:1], r, ref.gradient_bound(x[:1], r, g[:1]), form)
        assert not torch.isfinite(d[1, 5]) and torch.isnan(d[2]).all() and (d[3] == 0).all()


FIRST_CALL = """
import torch, reduction_pointwise_row_gb300 as fr
x = torch.randn(300, 40000, device="cuda").bfloat16()
t, g = torch.zeros(300, dtype=torch.int64, device="cuda"), torch.ones(1, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    a = fr.fr_logprobs(x, t, top=5, form="looped")
    b = fr.fr_xent_backward(x, t, g, form="persistent")
    c = fr.fr_logprobs(x, t, top=5, form="split")
graph.replay()
torch.cuda.synchronize()
assert torch.equal(a["top_index"], c["top_index"])
assert torch.equal(a["top_index"], x.float().topk(5).indices) or (x.float().gather(
    1, a["top_index"]) == x.float().topk(5).values).all()
assert torch.allclose(b["loss"], -a["logprob"], atol=1e-4)
assert fr.fr_check_device_error() == 0
"""


def test_the_first_call_of_a_process_inside_a_capture():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], capture_output=True, text=True,
                       timeout=300, cwd=root)
    assert r.returncode == 0, r.stdout + r.stderr


OFFSETS = [s * o for o in (1e6, 3e7, 1e9, 5e9, 1e12, 1e20, 1e29, 6e29, 1e38) for s in (1, -1)]


def offset_rows(cols, dtype):
    """Rows far from zero: all at one value (what a finite mask leaves of a row), spread
    around it as far as the type has values there, and partly masked by -inf."""
    base = torch.from_numpy(rng(cols, 9).normal(0.0, 3.0, cols))
    rows = []
    for o in OFFSETS:
        rows += [torch.full((cols,), o, dtype=torch.float64), base + o,
                 torch.where(torch.arange(cols) % 3 == 1, -math.inf, base + o)]
    return torch.stack(rows).float().to(DTYPES[dtype])


@FORWARD_FORMS
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [40, 1000, 9001])
def test_rows_far_from_zero(cols, dtype, form):
    skip_long(form, cols, dtype)
    x = offset_rows(cols, dtype)
    t = torch.zeros(x.shape[0], dtype=torch.int64)
    i = torch.tensor([[0, 2, 3]]).repeat(x.shape[0], 1)
    z = torch.tensor([[0.5, 1.0, -1.0]]).repeat(x.shape[0], 1)
    got = fr.fr_logprobs(x.cuda(), t.cuda(), top=9, form=form)
    loss, r = fr.fr_distill(x.cuda(), i.cuda(), z.cuda(), form=form), ref.distill(x, i, z)
    bound = loss_bound(x, r, i, z, 1.0)
    for n in range(x.shape[0]):
        s = slice(n, n + 1)
        what = f"{OFFSETS[n // 3]:g}, kind {n % 3}, {cols} {dtype}"
        check_logprobs(x[s], {k: o[s] for k, o in got.items()}, t[s], 9, what)
        ref.assert_near(loss[s], r[s], bound[s], f"{what} distill")


@BACKWARD_FORMS
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [40, 1000, 9001])
def test_gradients_of_rows_far_from_zero(cols, dtype, form):
    x = offset_rows(cols, dtype)
    rows = x.shape[0]
    t = torch.zeros(rows, dtype=torch.int64)
    g, h = upstream(rows, 1), upstream(rows, 2)
    i = torch.tensor([[0, 2, 3]]).repeat(rows, 1)
    z = torch.tensor([[0.5, 1.0, -1.0]]).repeat(rows, 1)
    d, _ = run_backward(fr.fr_logprobs_backward, x, (0, 0), (0, 0), form, token=t.cuda(),
                        dlogprob=g.cuda(), dentropy=h.cuda())
    e, loss = run_backward(fr.fr_xent_backward, x, (0, 0), (0, 0), form, target=t.cuda(),
                           dloss=g.cuda())
    k, _ = run_backward(fr.fr_distill_backward, x, (0, 0), (0, 0), form, teacher_index=i.cuda(),
                        teacher_logit=z.cuda(), dloss=g.cuda())
    rd, re, rk = (ref.logprobs_backward(x, t, g, h), ref.xent_backward(x, t, g),
                  ref.distill_backward(x, i, z, g))
    bd, be = ref.gradient_bound(x, rd, g, h), ref.gradient_bound(x, re, g)
    bk = ref.gradient_bound(x, rk, g) + g.double().abs()[:, None] * 160 * ref.U
    rl = ref.xent(x, t)
    for n in range(rows):
        s = slice(n, n + 1)
        what = f"{OFFSETS[n // 3]:g}, kind {n % 3}, {cols} {dtype}"
        ref.assert_near(d[s], rd[s], bd[s], f"{what} logprobs")
        ref.assert_near(e[s], re[s], be[s], f"{what} xent")
        ref.assert_near(k[s], rk[s], bk[s], f"{what} distill")
        ref.assert_near(loss[s], rl[s], ref.eps(cols) + 4 * ref.U * rl[s].abs(), f"{what} loss")


@pytest.mark.parametrize("temperature", [0.25, 0.5, 1.0])
def test_teacher_entries_at_the_lowest_value(temperature):
    """A masked element that the teacher gives weight costs its distance, which divided
    by a temperature below 1 is past fp32: the loss is not."""
    x = logits(6, 9000, "f32", 5)
    x[:, ::2] = torch.finfo(torch.float32).min
    i = torch.tensor([[0, 1, 3]]).repeat(6, 1)
    z = torch.tensor([[0.0, 1.0, 2.0]]).repeat(6, 1)
    r = ref.distill(x, i, z, temperature)
    # T q_0 3.4e38 with q_0 = exp(-2 / T) / sum: 2.8e34 at T = 1/4, 3.1e37 at 1
    assert (r > 1e34).all() and (r < 3e38).all()
    b = loss_bound(x, r, i, z, temperature)
    for form in ("looped", "split"):
        ref.assert_near(fr.fr_distill(x.cuda(), i.cuda(), z.cuda(), temperature, form=form), r, b)
    for form in ("looped", "persistent", "split"):
        got = fr.fr_distill_backward(x.cuda(), i.cuda(), z.cuda(), torch.ones(1, device="cuda"),
                                     temperature, form=form)
        ref.assert_near(got["loss"], r, b, form)


def test_a_workspace_with_gaps_is_refused():
    x = logits(700, 4099, "bf16", 1).cuda()
    n = fr.fr_workspace_size("logprobs", 700, 4099, "bf16")
    for ws in (torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2],
               torch.empty(1, dtype=torch.uint8, device="cuda").expand(n)):
        with pytest.raises(ValueError):
            fr.fr_logprobs(x, top=3, workspace=ws)


def test_a_gradient_between_the_logits_rows():
    """dlogits in the padding of the logits' rows."""
    both = torch.zeros(300, 2 * 12000, device="cuda")
    x, t = logits(300, 12000, "f32", 6), tokens(300, 12000, 6)
    both[:, :12000] = x.cuda()
    g = upstream(300, 6)
    r = ref.xent_backward(x, t, g)
    for form in ("looped", "persistent", "split"):
        d = fr.fr_xent_backward(both[:, :12000], t.cuda(), g.cuda(), dlogits=both[:, 12000:],
                                form=form)["dlogits"]
        ref.assert_near(d, r, ref.gradient_bound(x, r, g), form)
        assert torch.equal(both[:, :12000].cpu(), x)
    with pytest.raises(fr.FRError):
        fr.fr_xent_backward(both[:, :12000], t.cuda(), g.cuda(), dlogits=both[:, 11999:23999])


@pytest.mark.parametrize("temperature", [0.5, 0.99, 2.0])
def test_a_teacher_whose_entries_are_all_masked(temperature):
    """T 3.4e38 and a little: in range for T < 1, +inf for 2."""
    x = logits(3, 700, "f32", 5)
    x[:, :60] = torch.finfo(torch.float32).min
    i = torch.arange(50).repeat(3, 1)
    z = torch.from_numpy(rng(50).normal(0, 3, (3, 50)).astype(np.float32))
    r = ref.distill(x, i, z, temperature).float().double()
    b = loss_bound(x, r, i, z, temperature)
    assert torch.isinf(r).all() == (temperature > 1)
    for form in ("looped", "split", "persistent"):
        ref.assert_near(fr.fr_distill(x.cuda(), i.cuda(), z.cuda(), temperature, form=form), r, b)
        got = fr.fr_distill_backward(x.cuda(), i.cuda(), z.cuda(), torch.ones(1, device="cuda"),
                                     temperature, form=form)
        ref.assert_near(got["loss"], r, b, form)
