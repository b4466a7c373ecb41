"""The staged gradients over many rows a CTA or cluster, against the 64-bit formulas:
every ring of that form -- the rows' names, the answers to requests for another row, the
helpers' slots, the buffers (one of them too) and the cluster's statistics -- comes round
several times, with ignored rows, bad ones and rows without weight in between, out of
place and in place."""
import math

import pytest
import torch

import logits_ref as ref
import reduction_pointwise_row_gb300 as fr

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# (form, dtype, rows, cols): 152 SMs hold at most 608 CTAs of short rows, 152 of long ones
RINGS = [("persistent", "bf16", 25000, 9000),   # about 41 rows a CTA
         ("split", "bf16", 25000, 9000),        # clusters of 2: about 82 rows each
         ("persistent", "bf16", 5500, 65537),   # one buffer, 36 rows a CTA
         ("split", "bf16", 3000, 90001),        # clusters of 2, one CTA an SM
         ("auto", "bf16", 1400, 128256),        # clusters of 4, about 37 rows each
         ("auto", "bf16", 700, 262144),         # clusters of 8, about 37 rows each
         ("split", "f32", 700, 262145)]         # clusters of 8 with one buffer


def near(got, want, bound, what):
    """As ref.assert_near, on the GPU."""
    got = got.double()
    bound = bound.expand_as(want)
    for name, f in (("NaN", torch.isnan), ("inf", torch.isinf)):
        assert torch.equal(f(got), f(want)), f"{what}: {name} at other places"
    off = torch.where(torch.isfinite(want), (got - want).abs() - bound, -1.0)
    assert not bool((off > 0).any()), (what, torch.nonzero(off > 0)[0].tolist(), float(off.max()))


def slices(rows, cols):
    step = max(1, (1 << 25) // cols)
    return [slice(a, min(rows, a + step)) for a in range(0, rows, step)]


def made(rows, cols, dtype, seed):
    """Logits of row-dependent size, targets (some ignored, some bad) and upstream gradients."""
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.empty(rows, cols, dtype=DTYPES[dtype], device="cuda")
    x.normal_(0.0, 3.0, generator=g)
    x *= 0.5 + torch.rand(rows, 1, generator=g, device="cuda").to(x.dtype)
    u = torch.rand(rows, generator=g, device="cuda")
    t = torch.randint(0, cols, (rows,), generator=g, device="cuda")
    t[u < 0.1] = -100
    t[(u > 0.1) & (u < 0.13)] = cols
    t[(u > 0.13) & (u < 0.16)] = -1
    d = torch.randn(2, rows, generator=g, device="cuda")
    return g, x, t, d[0], d[1], u


def places(x):
    """(logits, dlogits or None): into a matrix of its own, and over the logits."""
    yield x, None
    y = x.clone()
    yield y, y


def rings(test):
    return pytest.mark.parametrize("form,dtype,rows,cols", RINGS)(test)


@rings
def test_cross_entropy(form, dtype, rows, cols):
    _, x, t, d, _, _ = made(rows, cols, dtype, 1)
    for v, out in places(x):
        r = fr.fr_xent_backward(v, t, d, dlogits=out, form=form)
        with torch.device("cuda"):
            for s in slices(rows, cols):
                want = ref.xent_backward(x[s], t[s], d[s])
                near(r["dlogits"][s], want, ref.gradient_bound(x[s], want, d[s]), f"rows {s}")
                loss = ref.xent(x[s], t[s])
                near(r["loss"][s], loss, ref.eps(cols) + 4 * ref.U * loss.abs(), f"loss {s}")
        assert fr.fr_check_device_error() == 1  # the bad targets


@rings
def test_log_probability_and_entropy(form, dtype, rows, cols):
    _, x, t, d, h, _ = made(rows, cols, dtype, 2)
    for v, out in places(x):
        r = fr.fr_logprobs_backward(v, t, d, h, dlogits=out, form=form)
        with torch.device("cuda"):
            for s in slices(rows, cols):
                want = ref.logprobs_backward(x[s], t[s], d[s], h[s])
                near(r[s], want, ref.gradient_bound(x[s], want, d[s], h[s]), f"rows {s}")
        assert fr.fr_check_device_error() == 1


def loss_bound(x, index, logit, temperature):
    """T^2 sum q (log q - log p): each log within EPS plus its own rounding."""
    _, _, logp, _ = ref.parts(x, temperature)
    q, logq, _ = ref.teacher(index, logit, temperature)
    at = logp.gather(1, index.clamp(0, x.shape[1] - 1))
    size = torch.nan_to_num(q * (logq.abs() + at.abs() + 1), nan=0.0, posinf=0.0).sum(1)
    return temperature ** 2 * size * (2 * ref.eps(x.shape[1]) + 160 * ref.U)


@rings
def test_distillation(form, dtype, rows, cols):
    temperature, top = 2.0, 40
    g, x, _, d, _, u = made(rows, cols, dtype, 3)
    i = torch.randint(0, cols, (rows, top), generator=g, device="cuda")
    i[torch.rand(rows, top, generator=g, device="cuda") < 0.2] = -1
    i[:, 5] = i[:, 4]             # repeats
    i[u < 0.1] = -1               # no weight
    i[(u > 0.1) & (u < 0.13), 7] = cols
    z = 3 * torch.randn(rows, top, generator=g, device="cuda")
    for v, out in places(x):
        r = fr.fr_distill_backward(v, i, z, d, temperature, dlogits=out, form=form)
        with torch.device("cuda"):
            for s in slices(rows, cols):
                want = ref.distill_backward(x[s], i[s], z[s], d[s], temperature)
                q, _, _ = ref.teacher(i[s], z[s], temperature)
                dense = torch.zeros_like(want).scatter_add_(1, i[s].clamp(0, cols - 1), q)
                bound = ref.gradient_bound(x[s], want, d[s] * temperature, temperature=temperature)
                # the entries' weights, each within 64 u of its share, add up at the size of g T
                bound += d[s].double().abs()[:, None] * temperature * dense * 160 * ref.U
                near(r["dlogits"][s], want, bound, f"rows {s}")
                near(r["loss"][s], ref.distill(x[s], i[s], z[s], temperature),
                     loss_bound(x[s], i[s], z[s], temperature), f"loss {s}")
        assert fr.fr_check_device_error() == 1


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
