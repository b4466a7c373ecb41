"""The calls over rows of logits, without a GPU: arguments refused on the host
before any CUDA call, and the 64-bit formulas that the GPU tests use against
automatic differentiation and independent library routines."""
import ctypes
import math

import pytest
import torch

import logits_ref as ref
import reduction_pointwise_row_gb300 as fr

P = ctypes.c_void_p
GOOD, ODD, HALF = P(0x10000), P(0x10001), P(0x10004)
OTHER = P(0x20000)
BIG = 1 << 40
OK_SO_FAR = 8  # every argument accepted: without a device, FR_ERR_NO_DEVICE


def logprobs(logits=GOOD, token=GOOD, logprob=GOOD, entropy=GOOD, lse=GOOD, tl=GOOD, ti=GOOD,
             top=4, rows=4, cols=8, ld=8, dtype=1, form=0):
    return fr.lib().fr_logprobs(logits, token, logprob, entropy, lse, tl, ti, top, rows, cols, ld,
                                -100, dtype, form, None, 0, None)


def logprobs_backward(logits=GOOD, token=GOOD, dlp=GOOD, dlps=1, dent=GOOD, dents=1,
                      dlogits=OTHER, rows=4, cols=8, ld=8, ldd=8, dtype=1, form=0):
    return fr.lib().fr_logprobs_backward(logits, token, dlp, dlps, dent, dents, dlogits, rows,
                                         cols, ld, ldd, -100, dtype, form, None)


def distill(logits=GOOD, index=GOOD, z=GOOD, loss=GOOD, top=4, rows=4, cols=8, ld=8, ldt=4,
            temperature=1.0, dtype=1, form=0):
    return fr.lib().fr_distill(logits, index, z, loss, top, rows, cols, ld, ldt, temperature,
                               dtype, form, None)


def distill_backward(logits=GOOD, index=GOOD, z=GOOD, dloss=GOOD, stride=1, loss=GOOD,
                     dlogits=OTHER, top=4, rows=4, cols=8, ld=8, ldd=8, ldt=4, temperature=1.0,
                     dtype=1, form=0):
    return fr.lib().fr_distill_backward(logits, index, z, dloss, stride, loss, dlogits, top, rows,
                                        cols, ld, ldd, ldt, temperature, dtype, form, None)


def xent_backward(logits=GOOD, target=GOOD, dloss=GOOD, stride=1, loss=GOOD, dlogits=OTHER,
                  rows=4, cols=8, ld=8, ldd=8, dtype=1, form=0):
    return fr.lib().fr_xent_backward(logits, target, dloss, stride, loss, dlogits, rows, cols, ld,
                                     ldd, -100, dtype, form, None)


SHARED = [(dict(logits=None), 1), (dict(rows=0), 1), (dict(cols=0), 1), (dict(rows=-1), 1),
          (dict(ld=7), 1), (dict(dtype=2), 2), (dict(dtype=-1), 2), (dict(logits=ODD), 4),
          (dict(logits=P(0x10002), dtype=0), 4), (dict(form=9), 3),
          (dict(rows=BIG, cols=BIG, ld=BIG), 1)]
GRADIENT = [(dict(dlogits=None), 1), (dict(ldd=7), 1), (dict(dlogits=ODD), 4),
            (dict(dlogits=GOOD, ldd=16), 1), (dict(rows=BIG, ldd=BIG), 1)]
TEACHER = [(dict(index=None), 1), (dict(z=None), 1), (dict(top=0), 1), (dict(top=129), 1),
           (dict(ldt=3), 1), (dict(temperature=0.0), 1), (dict(temperature=-2.0), 1),
           (dict(temperature=math.inf), 1), (dict(temperature=math.nan), 1),
           (dict(temperature=1e-39), 1), (dict(index=HALF), 4), (dict(z=ODD), 4),
           (dict(rows=BIG, ldt=BIG), 1)]
UPSTREAM = [(dict(dloss=None), 1), (dict(stride=-1), 1), (dict(stride=BIG, rows=BIG), 1),
            (dict(dloss=ODD), 4), (dict(loss=ODD), 4)]
CASES = [
    (logprobs, SHARED + [(dict(top=-1), 1), (dict(top=9), 1), (dict(top=129, cols=200, ld=200), 1),
                         (dict(top=0), 1), (dict(tl=None), 1), (dict(ti=None), 1),
                         (dict(token=None), 1), (dict(token=HALF), 4), (dict(logprob=ODD), 4),
                         (dict(entropy=ODD), 4), (dict(lse=ODD), 4), (dict(tl=ODD), 4),
                         (dict(ti=HALF), 4),
                         (dict(logprob=None, entropy=None, lse=None, tl=None, ti=None, top=0), 1)]),
    (logprobs_backward, SHARED + GRADIENT + [
        (dict(dlp=None, dent=None), 1), (dict(token=None), 1), (dict(token=HALF), 4),
        (dict(dlp=ODD), 4), (dict(dent=ODD), 4), (dict(dlps=-1), 1), (dict(dents=-1), 1),
        (dict(dents=BIG, rows=BIG), 1)]),
    (distill, SHARED + TEACHER + [(dict(loss=None), 1), (dict(loss=ODD), 4)]),
    (distill_backward, SHARED + GRADIENT + TEACHER + UPSTREAM),
    (xent_backward, SHARED + GRADIENT + UPSTREAM + [(dict(target=None), 1), (dict(target=HALF), 4)]),
]


@pytest.mark.parametrize("call,cases", CASES, ids=[c.__name__ for c, _ in CASES])
def test_arguments_are_refused_on_the_host(call, cases):
    for kw, status in cases:
        assert call(**kw) == status, (call.__name__, kw)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are not device memory")
def test_accepted_arguments_reach_the_device_check():
    assert logprobs() == OK_SO_FAR
    assert logprobs(token=None, logprob=None, top=0, tl=None, ti=None) == OK_SO_FAR
    assert logprobs_backward(token=None, dlp=None) == OK_SO_FAR
    assert logprobs_backward(dent=None, dlogits=GOOD) == OK_SO_FAR
    assert distill(ldt=9) == OK_SO_FAR
    assert distill_backward(stride=0, loss=None) == OK_SO_FAR
    assert xent_backward(stride=0, loss=None, dlogits=GOOD, dtype=0) == OK_SO_FAR


def test_the_binding_refuses_host_tensors():
    x, t, g = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64), torch.ones(4)
    i, z = torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2)
    for call in (lambda: fr.fr_logprobs(x, t), lambda: fr.fr_logprobs_backward(x, t, g),
                 lambda: fr.fr_distill(x, i, z), lambda: fr.fr_distill_backward(x, i, z, g),
                 lambda: fr.fr_xent_backward(x, t, g)):
        with pytest.raises(ValueError):
            call()


def test_formulas_against_automatic_differentiation():
    torch.manual_seed(1)
    x = (3 * torch.randn(6, 50, dtype=torch.float64)).requires_grad_()
    t = torch.tensor([1, -100, 3, 49, 0, 7])
    g, h = torch.randn(6), torch.randn(6)
    lp = torch.log_softmax(x, 1)
    at = torch.where(t == -100, 0.0, lp.gather(1, t.clamp(min=0)[:, None])[:, 0])
    entropy = torch.distributions.Categorical(logits=x).entropy()
    r = ref.logprobs(x.detach(), t, 5)
    assert torch.allclose(r["logprob"], at, atol=1e-12)
    assert torch.allclose(r["entropy"], entropy, atol=1e-12)
    assert torch.allclose(r["lse"], torch.logsumexp(x, 1), atol=1e-12)
    assert torch.equal(r["top_index"], torch.topk(x, 5).indices)
    (at * g + entropy * h).sum().backward()
    assert torch.allclose(x.grad, ref.logprobs_backward(x.detach(), t, g, h), atol=1e-12)

    x.grad = None
    loss = torch.nn.functional.cross_entropy(x, t, reduction="none", ignore_index=-100)
    assert torch.allclose(loss, ref.xent(x.detach(), t), atol=1e-12)
    (loss * g).sum().backward()
    assert torch.allclose(x.grad, ref.xent_backward(x.detach(), t, g), atol=1e-12)

    x.grad = None
    temperature = 1.7
    i = torch.stack([torch.randperm(50)[:6] for _ in range(6)])
    i[2, 1] = i[2, 0]
    z = torch.randn(6, 6, dtype=torch.float64)
    q = torch.softmax(z / temperature, 1)
    logp = torch.log_softmax(x / temperature, 1).gather(1, i)
    loss = temperature ** 2 * (q * (q.log() - logp)).sum(1)
    assert torch.allclose(loss, ref.distill(x.detach(), i, z, temperature), atol=1e-12)
    (loss * g).sum().backward()
    assert torch.allclose(x.grad, ref.distill_backward(x.detach(), i, z, g, temperature), atol=1e-12)


def test_the_comparison_notices_mistakes():
    """A formula with a planted mistake is outside the bounds: no ignored rows, the
    padding entries counted, the temperature left out of the gradient, entropy
    about the wrong mean, ties to the higher index."""
    torch.manual_seed(2)
    x = (3 * torch.randn(5, 300)).bfloat16()
    t = torch.tensor([1, -100, 3, 299, 0])
    g = torch.ones(5)
    i = torch.randint(0, 300, (5, 4))
    i[:, 3] = -1
    z = torch.randn(5, 4)

    def differs(wrong, right, bound):
        with pytest.raises(AssertionError):
            ref.assert_near(wrong, right, bound)

    right = ref.xent_backward(x, t, g)
    differs(ref.xent_backward(x, t.clamp(min=0), g), right, ref.gradient_bound(x, right, g))
    right = ref.distill_backward(x, i, z, g, 2.0)
    bound = ref.gradient_bound(x, right, 2 * g, temperature=2.0)
    differs(ref.distill_backward(x, i.clamp(min=0), z, g, 2.0), right, bound)
    differs(ref.distill_backward(x, i, z, g, 2.0) / 2, right, bound)
    right = ref.logprobs_backward(x, None, None, g)
    _, _, logp, p = ref.parts(x)
    differs(-p * logp, right, ref.gradient_bound(x, right, torch.zeros(1), g))
    tied = torch.zeros(1, 9)
    assert ref.logprobs(tied, None, 3)["top_index"].tolist() == [[0, 1, 2]]
    tied[0, 4] = math.nan
    tied[0, 6] = math.inf
    assert ref.logprobs(tied, None, 3)["top_index"].tolist() == [[4, 6, 0]]


def test_the_forms_that_auto_takes():
    """Host-side rules: a warp per short row, a cluster per long one, a CTA per row for
    few rows, and never a form past its limits."""
    def form(op, rows, cols, dtype="bf16"):
        return fr.fr_auto_form(op, rows, cols, dtype, 152)

    for op in ("logprobs", "distill"):
        assert form(op, 4000, 1000) == "persistent" and form(op, 1, 50257) == "split"
        assert form(op, 8192, 50257) == "looped"
    assert form("logprobs", 700, 50257) == "looped" and form("distill", 700, 50257) == "split"
    for op in ("logprobs_backward", "distill_backward", "xent_backward"):
        assert form(op, 30000, 1000) == "persistent" and form(op, 4096, 50257) == "persistent"
        assert form(op, 8, 50257) == "looped" and form(op, 1024, 65537) == "split"
        assert form(op, 1024, 900000) in ("split", "looped")
        assert form(op, 4, 1 << 30) == "looped" and form(op, (1 << 31), 60000) == "looped"


def test_algorithmic_bytes_of_the_logits_calls():
    """Logits read once (and their gradient written once), plus the rows' vectors."""
    from reduction_pointwise_row_gb300 import traffic as t
    R, C = 7, 1001
    assert t.algorithmic_bytes("logprobs", R, C) == R * (2 * C + 20)
    assert t.algorithmic_bytes("logprobs", R, C, dtype="f32", top=5) == R * (4 * C + 20 + 60)
    assert t.algorithmic_bytes("logprobs_backward", R, C) == R * (4 * C + 16)
    assert t.algorithmic_bytes("distill", R, C, top=64) == R * (2 * C + 768 + 4)
    assert t.algorithmic_bytes("distill_backward", R, C, top=64) == R * (4 * C + 768 + 8)
    assert t.algorithmic_bytes("distill_backward", R, C, top=64, loss=False) == R * (4 * C + 772)
    assert t.algorithmic_bytes("xent_backward", R, C, dtype="f32") == R * (8 * C + 16)


OVERLAPS = [  # (dlogits - logits in bytes, rows, cols, ld, ldd, allowed), bf16
    (0, 4, 8, 8, 8, True), (0, 4, 8, 16, 8, False), (0, 4, 8, 8, 16, False),
    (0, 1, 8, 16, 8, True),
    (64, 4, 8, 8, 8, True), (62, 4, 8, 8, 8, False), (-64, 4, 8, 8, 8, True),
    (-62, 4, 8, 8, 8, False), (2, 4, 8, 8, 8, False), (16, 4, 8, 8, 8, False),
    (16, 4, 8, 16, 16, True), (14, 4, 8, 16, 16, False), (18, 4, 8, 16, 16, False),
    (-16, 4, 8, 16, 16, True), (-18, 4, 8, 16, 16, False), (48, 4, 8, 16, 16, True),
    (-80, 4, 8, 16, 16, True), (32, 4, 8, 16, 16, False), (16, 4, 8, 32, 16, False),
    (16, 4, 8, 20, 20, True), (24, 4, 8, 20, 20, True), (26, 4, 8, 20, 20, False),
    (8, 1, 8, 100, 100, False), (16, 1, 8, 8, 8, True), (-16, 1, 8, 8, 8, True),
]


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are not device memory")
@pytest.mark.parametrize("shift,rows,cols,ld,ldd,allowed", OVERLAPS)
def test_gradients_over_a_part_of_the_logits_are_refused(shift, rows, cols, ld, ldd, allowed):
    used = {(r * ld + j) * 2 for r in range(rows) for j in range(cols)}
    own = {shift + (r * ldd + j) * 2 for r in range(rows) for j in range(cols)}
    if allowed:  # what is allowed is disjoint or the same rows
        assert not used & own or used == own
    for call in (logprobs_backward, distill_backward, xent_backward):
        assert call(dlogits=P(0x10000 + shift), rows=rows, cols=cols, ld=ld, ldd=ldd) == (
            OK_SO_FAR if allowed else 1)
