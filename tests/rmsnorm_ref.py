"""A residual block's row operators in 64 bits, and how far fp32 kernels may be off.

The dropout mask is generated with numpy's 64-bit integers from the published
definition of Philox4x32 (Salmon et al., "Parallel random numbers: as easy as 1, 2,
3", SC 2011).
"""
import numpy as np
import torch

U = 2.0 ** -24  # half an fp32 step, relative
E4M3_MAX = 448.0


def half_step(dtype):
    """Most a rounding to `dtype` is off, relative to the value."""
    return torch.finfo(dtype).eps / 2


def philox(ctr, key, rounds):
    """Philox4x32: ctr and key sequences of uint32 arrays (or ints) -> four uint32 arrays."""
    c = [np.asarray(v, np.uint64) for v in ctr]
    k = [int(v) for v in key]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) % 2**32, (k[1] + 0xBB67AE85) % 2**32]
    return [v.astype(np.uint32) for v in c]


def threshold(p):
    """How many of 65536 values of an element's 16 bits drop it."""
    p = float(np.float32(p))
    return 65536 if p == 1.0 else min(max(round(65536 * p), 1), 65535) if p else 0


def keep(rows, cols, p, rng, site=0):
    """(bool [rows, cols], factor): what stays, and what it is multiplied by."""
    seed, offset = (int(v) % 2**64 for v in rng)
    offset = (offset + site) % 2**64
    r, b = np.meshgrid(np.arange(rows), np.arange((cols + 7) // 8), indexing="ij")
    zero = np.zeros_like(r)
    words = philox([b, r, zero + offset % 2**32, zero + offset // 2**32],
                   [seed % 2**32, seed // 2**32], 7)
    halves = np.stack([h for w in words for h in (w & 0xFFFF, w >> 16)], 2).reshape(rows, -1)
    t = threshold(p)
    return (torch.from_numpy((halves[:, :cols] >= t)),
            65536.0 / (65536 - t) if t < 65536 else 0.0)


def dropout(x, p, rng, site=0, residual=None):
    v = x.double()
    if p:
        m, f = keep(*x.shape, p, rng, site)
        v = torch.where(m, v * f, 0.0)
    return v if residual is None else v + residual.double()


def dropout_bound(x, p, residual, want, dtype):
    """The factor's and the product's rounding, the addition's, and the output's."""
    f = 65536.0 / (65536 - threshold(p)) if 0 < threshold(p) < 65536 else 1.0
    size = x.double().abs() * f + (0.0 if residual is None else residual.double().abs())
    return 3 * U * size + half_step(dtype) * want.abs() * (1 + 4 * U) + tiny(dtype)


def tiny(dtype):
    """Half the smallest step of a type near zero."""
    return {torch.bfloat16: 2.0**-134, torch.float32: 2.0**-150}[dtype]


def norm(h, gamma, eps):
    """(y, rstd) in 64 bits."""
    h = h.double()
    rstd = 1.0 / torch.sqrt(h.square().mean(1) + eps)
    return h * rstd[:, None] * gamma.double(), rstd


def sum_depth(cols):
    """Additions that a term of a row's sum goes through, at most: 32 of a lane (or 8 of
    a chunk and the chunks of a lane of the looped form), 5 levels within a warp and 5
    over warps."""
    return 32 + 8 + -(-cols // 4096) + 10


def rstd_bound(cols):
    """Relative: half the sum's (its terms are positive; each square one rounding more),
    and the quotient's, eps' addition, the root's and the reciprocal's."""
    return ((sum_depth(cols) + 1) / 2 + 4) * U


def norm_bound(cols, want, dtype):
    """rstd's, two products', the output's."""
    return (rstd_bound(cols) + 2 * U) * 1.01 * want.abs() + half_step(dtype) * want.abs() * \
        (1 + 2 * rstd_bound(cols)) + tiny(dtype)


def groups_of(v, width):
    """[rows, groups, width] of v [rows, cols], zeros past the last column."""
    rows, cols = v.shape
    g = -(-cols // width)
    full = torch.zeros(rows, g * width, dtype=v.dtype)
    full[:, :cols] = v
    return full.view(rows, g, width)


def scales(v, width):
    """[rows, groups]: the largest magnitude over each `width` columns / 448."""
    return (groups_of(v, width).abs().amax(2) / E4M3_MAX).clamp(min=2.0**-126)


def quant_bound(cols, v, scale):
    """Of y8 * scale, given the scale that was used: e4m3's half step (2^-4 relative, at
    least half of 2^-9) of what fp32 gave."""
    e = rstd_bound(cols) + 4 * U
    return v.abs() * (2.0**-4 * (1 + 2 * e) + e) + scale * 2.0**-10


def backward(dy, h, gamma, rstd, dh=None):
    """(dresidual, dgamma) in 64 bits."""
    dy, n = dy.double(), h.double() * rstd.double()[:, None]
    u = dy * gamma.double()
    d = rstd.double()[:, None] * (u - n * (u * n).mean(1, keepdim=True))
    return d if dh is None else d + dh.double(), (dy * n).sum(0)


def backward_bound(dy, h, gamma, rstd, dh, want, dtype):
    """mean(u n): each product two or three roundings, the sum's depth, three factors; then
    n, u, the fused difference, the product with rstd and dh's addition; the output."""
    r = rstd.double()[:, None]
    n, u = h.double().abs() * r, (dy.double() * gamma.double()).abs()
    mean = (u * n).mean(1, keepdim=True)
    e = r * (n * mean * (sum_depth(h.shape[1]) + 9) + u * 4 + n * mean * 4) * U
    if dh is not None:
        e = e + dh.double().abs() * U + want.abs() * U
    return 1.01 * e + half_step(dtype) * (want.abs() + e) + tiny(dtype)


def dgamma_bound(dy, h, rstd):
    """Each term two roundings, and a rounding an addition: of the rows in turn, of a CTA's
    row groups (at most 8), of the shares (a 32nd of them, in turn) and 5 levels."""
    t = (dy.double() * h.double() * rstd.double()[:, None]).abs().sum(0)
    return (2 + dy.shape[0] + 8 + 5) * U * 1.01 * t + 2.0**-149


def assert_near(got, want, bound, what=""):
    g, w = got.detach().cpu().double(), want.double()
    assert g.shape == w.shape, what
    b = torch.as_tensor(bound, dtype=torch.float64).expand(w.shape)
    assert torch.equal(g.isnan(), w.isnan()), f"{what}: NaN in other places"
    ok = (g - w).abs() <= b
    ok |= (g == w) | w.isnan()
    if not ok.all():
        i = ((g - w).abs() / b.clamp(min=1e-300)).nan_to_num(0.0).where(~ok, 0.0).argmax()
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.numel()} off, the worst at {int(i)}: "
                             f"{float(g.flatten()[i])!r} for {float(w.flatten()[i])!r}, bound "
                             f"{float(b.flatten()[i])!r}")
