"""Plain 64-bit formulas of the calls over rows of logits, and how far the
kernels' results may be from them.

Bounds.  With u = 2^-24 (half a step of fp32), t = (x - m) log2(e) / T:
  * exp((x - m) / T) is ex2 of t: ex2.approx is within 2^-22 relative, t carries two
    roundings and c = log2(e) / T two more, 4 u |t| of relative error, and where
    the exponential is below 2^-126 it is 0;
  * l and s are sums whose longest chain of additions is 64 + cols / 4096 long
    (up to 32 per group of vectors, one per group, the merges of 32 lanes and of at most
    32 warps and 16 CTAs, each of three roundings and one ex2): chain(cols) u + 14 *
    2^-22 relative of the sum of magnitudes.
So log l is within EPS = (64 + cols / 4096 + 64) u + 2^-18 absolute, which also
covers the E|t| 4 u of the exponentials (E|t| <= 20), and what follows from l and
the roundings of the formulas is counted in EPS, below.  A bf16 result adds half a step, 2^-8 relative.
"""
import math

import torch

U = 2.0 ** -24
TINY = 2.0 ** -120  # what flushed exponentials may miss, per unit of the factors


def eps(cols: int) -> float:
    return (128 + cols / 4096) * U + 2.0 ** -18


def parts(x, temperature=1.0):
    """(m, d, logp, p) in fp64; x - m of -inf logits is -inf."""
    x = x.double()
    m = x.amax(1, keepdim=True)
    d = x - m
    logp = d / temperature - torch.log(torch.exp(d / temperature).sum(1, keepdim=True))
    return m, d, logp, torch.exp(logp)


def _xlogx(p, logp):
    return torch.where(p > 0, p * logp, torch.where(torch.isnan(p), p, torch.zeros_like(p)))


def logprobs(x, token=None, top=0, ignore_index=-100):
    m, d, logp, p = parts(x)
    cols = x.shape[1]
    o = {"entropy": -_xlogx(p, logp).sum(1),
         "lse": torch.where(m == -math.inf, m, m + torch.log(
             torch.exp(d).sum(1, keepdim=True)))[:, 0]}
    if token is not None:
        good = (token >= 0) & (token < cols)
        lp = logp.gather(1, token.clamp(0, cols - 1)[:, None])[:, 0]
        lp = torch.where(good, lp, math.nan)
        o["logprob"] = torch.where(token == ignore_index, 0.0, lp)
    if top:
        key = torch.where(torch.isnan(x), math.inf, x.double())
        # NaN above +inf: a second key breaks that tie before the index does
        nan = torch.isnan(x).to(torch.int8)
        order = torch.argsort(key, dim=1, descending=True, stable=True)
        order = order.gather(1, torch.argsort(nan.gather(1, order), dim=1, descending=True,
                                              stable=True))
        o["top_index"] = order[:, :top]
        o["top_logprob"] = logp.gather(1, o["top_index"])
    return o


def teacher(index, logit, temperature):
    live = index >= 0
    z = torch.where(live, logit.double() / temperature, -math.inf)
    m = z.amax(1, keepdim=True)
    weight = (m != -math.inf)[:, 0]
    d = torch.where(weight[:, None], z - m, -math.inf)
    logq = d - torch.log(torch.exp(d).sum(1, keepdim=True).clamp(min=1e-300))
    q = torch.where(weight[:, None], torch.exp(logq), 0.0)
    return q, logq, weight


def distill(x, index, logit, temperature=1.0):
    cols = x.shape[1]
    _, _, logp, _ = parts(x, temperature)
    q, logq, weight = teacher(index, logit, temperature)
    at = logp.gather(1, index.clamp(0, cols - 1))
    term = torch.where(q == 0, 0.0, q * (logq - at))
    loss = temperature ** 2 * term.sum(1)
    loss = torch.where(weight, loss, 0.0)
    return torch.where((index >= cols).any(1), math.nan, loss)


def distill_backward(x, index, logit, dloss, temperature=1.0):
    cols = x.shape[1]
    _, _, _, p = parts(x, temperature)
    q, _, weight = teacher(index, logit, temperature)
    dense = torch.zeros_like(p).scatter_add_(1, index.clamp(0, cols - 1), q)
    g = dloss.double().expand(x.shape[0])[:, None] * temperature
    dx = torch.where(weight[:, None], g * (p - dense), 0.0)
    return torch.where((index >= cols).any(1)[:, None], math.nan, dx)


def logprobs_backward(x, token=None, dlogprob=None, dentropy=None, ignore_index=-100):
    rows, cols = x.shape
    _, d, logp, p = parts(x)
    dx = torch.zeros(rows, cols, dtype=torch.float64)
    if dlogprob is not None:
        hit = token != ignore_index
        bad = hit & ((token < 0) | (token >= cols))
        onehot = torch.zeros_like(dx).scatter_(1, token.clamp(0, cols - 1)[:, None], 1.0)
        g = torch.where(hit, dlogprob.double().expand(rows), 0.0)[:, None]
        dx = torch.where(hit[:, None], g * (onehot - p), 0.0)
        dx = torch.where(bad[:, None], math.nan, dx)
    if dentropy is not None:
        plogp = _xlogx(p, logp)
        h = dentropy.double().expand(rows)[:, None]
        dx = dx - h * (plogp - p * plogp.sum(1, keepdim=True))
    return dx


def xent(x, target, ignore_index=-100):
    return -logprobs(x, target, ignore_index=ignore_index)["logprob"] + 0.0


def xent_backward(x, target, dloss, ignore_index=-100):
    return logprobs_backward(x, target, -dloss, ignore_index=ignore_index)


# ---- comparison ---------------------------------------------------------------

def assert_near(got, ref, bound, what=""):
    """NaN and infinities where the formula has them; else |got - ref| <= bound."""
    got, ref = got.detach().cpu().double(), ref.double()
    bound = torch.as_tensor(bound, dtype=torch.float64).expand_as(ref)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    for name, f in (("NaN", torch.isnan), ("inf", torch.isinf)):
        assert torch.equal(f(got), f(ref)), f"{what}: {name} at other places"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities of the other sign"
    fin = torch.isfinite(ref)
    err, lim = (got - ref).abs()[fin], bound[fin]
    if err.numel() and not bool((err <= lim).all()):
        i = int(torch.argmax(err / lim))
        at = torch.nonzero(fin)[i].tolist()
        raise AssertionError(f"{what}: at {at} got {got[fin][i]:.9g}, formula {ref[fin][i]:.9g}, "
                             f"off by {err[i]:.3g}, bound {lim[i]:.3g}")


def gradient_bound(x, ref, g, h=None, temperature=1.0):
    """For dx = g (delta - p) - h p (log p + H) and its relatives: p is within
    (2 EPS + 8 u |t|) relative, the sum with delta rounds at the size of g, the
    entropy's factor is within EPS (2 + |log p + H| + H), H <= log cols."""
    cols = x.shape[1]
    e = eps(cols)
    _, d, logp, p = parts(x, temperature)
    t = torch.nan_to_num(d, neginf=0.0).abs() / temperature
    rel = 2 * e + 8 * U * t
    g = g.double().abs().expand(x.shape[0])[:, None]
    big = (ref.abs() > 0.0) | (p > 0)
    bound = g * (p * rel + TINY) + 4 * U * torch.where(big, g * (p + (ref.abs() > p * g / 2)), 0.0)
    if h is not None:
        far = torch.nan_to_num(logp, neginf=0.0).abs()
        bound = bound + h.double().abs().expand(x.shape[0])[:, None] * (
            p * (rel * (far + math.log(cols) + 1) + e * (2 + far + 2 * math.log(cols))) + TINY)
    bound = bound + 2 * U * ref.abs()
    if x.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * ref.abs() + 2.0 ** -133
    return torch.nan_to_num(bound, nan=0.0)
