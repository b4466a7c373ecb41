"""Measured cases of the row operators of a residual block: dropout whose mask
comes from a counter-based generator and is never stored, the root-mean-square
norm with the residual's addition, the same with an output in 8 bits and its
scales, and the norm's backward pass.

``listed()`` and ``draw()`` give the cases, ``prepare()`` makes a case's inputs
on the GPU from a seed, ``run()`` computes one pass -- in elementary torch
operations where ``own`` is false, through the library's calls where it is true
-- and ``exact()`` gives the same outputs in 64 bits.

The mask: element (r, c) is dropped where the 16-bit half e = c mod 8 of the
Philox4x32 block (7 rounds; Salmon et al., "Parallel random numbers: as easy as
1, 2, 3", SC 2011) with counter (c / 8, r, low and high word of offset + site)
and key (low and high word of seed) is less than t, t being 65536 p rounded and
at least 1; what stays is divided by 1 - t / 65536.
"""
import math

import numpy as np
import torch

own = False

OPS = ("rmsnorm", "rmsnorm", "rmsnorm_quant", "rmsnorm_backward", "dropout")
E4M3_MAX = 448.0
SITE = 3  # the place in the model whose mask is drawn


def _case(name, op, rows, cols, dtype="bf16", ld=0, residual=False, p=0.0, scale=""):
    """ld: distance between row starts (0: cols); residual: a residual is added before
    the norm (backward: a gradient reaches the sum by the residual's path too); p:
    dropout's probability; scale: "row", "group" (of 128 columns) or "given"."""
    c = dict(op=op, rows=rows, cols=cols, dtype=dtype, ld=max(ld, cols), residual=residual, p=p,
             scale=scale)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decoded token of one request: latency
        _case("norm_decode_1", "rmsnorm", 1, 8192, residual=True),
        # a pre-norm block of a training step: the branch's output dropped, added, normed
        _case("norm_train_16384", "rmsnorm", 16384, 4096, residual=True, p=0.1),
        # a narrow model's norm before its output head, no residual
        _case("norm_narrow_32768", "rmsnorm", 32768, 768),
        # an odd row length in fp32
        _case("norm_odd_f32_2047", "rmsnorm", 2047, 4097, "f32"),
        # a decode step of a batch before an 8-bit product with scales per 128 columns
        _case("quant_decode_61", "rmsnorm_quant", 61, 5120, residual=True, scale="group"),
        # a prefill before an 8-bit product with a scale per token
        _case("quant_prefill_8192", "rmsnorm_quant", 8192, 8192, residual=True, scale="row"),
        # calibrated activations: one given scale
        _case("quant_given_2048", "rmsnorm_quant", 2048, 10240, scale="given"),
        # the backward pass of norm_train_16384
        _case("norm_bwd_16384", "rmsnorm_backward", 16384, 4096, residual=True, p=0.1),
        # a wider model without dropout
        _case("norm_bwd_4096", "rmsnorm_backward", 4096, 8192, residual=True),
        # a small micro-batch in fp32
        _case("norm_bwd_33_f32", "rmsnorm_backward", 33, 1000, "f32"),
        # dropout alone: embeddings, and the backward pass of any dropout
        _case("dropout_16384", "dropout", 16384, 4096, p=0.1),
        # dropout and the residual's addition on an odd fp32 shape
        _case("dropout_odd_f32_1023", "dropout", 1023, 4099, "f32", residual=True, p=0.25),
    ]


def draw(rng):
    op = rng.choice(OPS)
    dtype = rng.choice(("bf16", "bf16", "f32"))
    cols = int(math.exp(rng.uniform(math.log(32), math.log(20000))))
    if rng.random() < 0.6:
        cols = max(8, cols // 8 * 8)
    most = 6.4e7 / cols / (2 if dtype == "f32" else 1)
    rows = max(1, int(math.exp(rng.uniform(0.0, math.log(min(16384.0, most))))))
    ld = cols + rng.choice((0, 0, 0, 8 * rng.randint(1, 8), rng.randint(1, 64)))
    p = rng.choice((0.0, 0.1, 0.25, 0.5))
    if op == "dropout":
        p = p or 0.05
    return _case("", op, rows, cols, dtype, ld, rng.random() < 0.7, p,
                 rng.choice(("row", "group", "given")) if op == "rmsnorm_quant" else "")


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    rows, cols, ld, op = (case[n] for n in ("rows", "cols", "ld", "op"))
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16

    def matrix(std, channels=False):
        buf = torch.empty(rows, ld, dtype=dt, device="cuda").normal_(0.0, std, generator=g)
        if channels:  # a residual stream has a few channels far larger than the others
            big = torch.randint(0, cols, (3,), generator=g, device="cuda")
            buf[:, big] *= 20.0
        return buf[:, :cols]

    st = dict(case, eps=1e-5)
    if op == "rmsnorm_backward":
        st["dy"] = matrix(0.02)
        h = matrix(2.0, True)
        st["dh"] = matrix(0.02) if case["residual"] else None
        st["h"] = h
        st["rstd"] = torch.rsqrt(h.double().square().mean(1) + st["eps"]).float()
    else:
        st["x"] = matrix(1.0)
        st["res"] = matrix(2.0, True) if case["residual"] else None
    if op != "dropout":
        st["gamma"] = 1.0 + 0.2 * torch.randn(cols, generator=g, device="cuda")
    st["rng"] = torch.randint(0, 2**63 - 1, (2,), generator=g, device="cuda") if case["p"] else None
    if case["scale"] == "given":
        st["given"] = 0.01 + 0.005 * torch.rand(1, generator=g, device="cuda")
    return st


def run(st):
    op, p, site = st["op"], st["p"], SITE
    if own:
        import reduction_pointwise_row_gb300 as fr
        if op == "dropout":
            return fr.fr_dropout(st["x"], p, st["rng"], site, residual=st["res"])
        if op == "rmsnorm":
            return fr.fr_rmsnorm(st["x"], st["gamma"], st["eps"], residual=st["res"], p=p,
                                 rng=st["rng"], site=site)
        if op == "rmsnorm_quant":
            scale = st["given"] if st["scale"] == "given" else st["scale"]
            return fr.fr_rmsnorm_quant(st["x"], st["gamma"], st["eps"], scale=scale,
                                       residual=st["res"], p=p, rng=st["rng"], site=site)
        return fr.fr_rmsnorm_backward(st["dy"], st["h"], st["gamma"], st["rstd"], dh=st["dh"], p=p,
                                      rng=st["rng"], site=site)
    if op == "rmsnorm_backward":
        return _plain_backward(st)
    x = st["x"]
    dt = x.dtype
    s = x.float()
    if p:
        keep, scale = _keep(st["rng"], p, *x.shape)
        s = torch.where(keep, s * scale, 0.0)
    if st["res"] is not None:
        s = s + st["res"].float()
    if op == "dropout":
        return s.to(dt)
    out = {}
    if p or st["res"] is not None:
        out["h"] = s.to(dt)
        s = out["h"].float()  # the norm is that of what the residual's path keeps
    rstd = torch.rsqrt(s.square().mean(1, keepdim=True) + st["eps"])
    y = s * rstd * st["gamma"]
    if op == "rmsnorm":
        out["rstd"] = rstd[:, 0]
        out["y"] = y.to(dt)
        return out
    if st["scale"] == "given":
        out["y"] = (y / st["given"]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return out
    rows, cols = y.shape
    width = cols if st["scale"] == "row" else 128
    groups = -(-cols // width)
    full = y.new_zeros(rows, groups * width)
    full[:, :cols] = y
    full = full.view(rows, groups, width)
    scale = (full.abs().amax(2) / E4M3_MAX).clamp(min=2.0**-126)
    q = (full / scale[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(rows, -1)[:, :cols]
    out["y"] = q.to(torch.float8_e4m3fn)
    out["scale"] = scale[:, 0] if st["scale"] == "row" else scale
    return out


def _threshold(p):
    return min(max(round(65536 * float(np.float32(p))), 1), 65535)


def _keep(rng, p, rows, cols):
    """The elements that stay, and their factor."""
    mask = 0xFFFFFFFF
    offset = rng[1] + SITE
    blocks = -(-cols // 8)
    c0 = torch.arange(blocks, device="cuda").expand(rows, blocks)
    c1 = torch.arange(rows, device="cuda")[:, None]
    c2, c3 = offset & mask, (offset >> 32) & mask
    k0, k1 = rng[0] & mask, (rng[0] >> 32) & mask
    for _ in range(7):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & mask) ^ c1 ^ k0, b & mask, ((a >> 32) & mask) ^ c3 ^ k1, a & mask
        k0, k1 = (k0 + 0x9E3779B9) & mask, (k1 + 0xBB67AE85) & mask
    words = torch.stack([h for w in (c0, c1, c2, c3) for h in (w & 0xFFFF, w >> 16)], 2)
    t = _threshold(p)
    keep = words.view(rows, 8 * blocks)[:, :cols] >= t
    return keep, 65536.0 / (65536 - t)


def _plain_backward(st):
    h, dt = st["h"].float(), st["dy"].dtype
    dy, rstd = st["dy"].float(), st["rstd"][:, None]
    w = dy * st["gamma"]
    c = (w * h).mean(1, keepdim=True)
    d = rstd * w - h * (rstd * rstd * rstd * c)
    if st["dh"] is not None:
        d = d + st["dh"].float()
    out = {"dgamma": (dy * (h * rstd)).sum(0)}
    if st["p"]:
        out["dresidual"] = d.to(dt)
        keep, scale = _keep(st["rng"], st["p"], *dy.shape)
        d = torch.where(keep, d * scale, 0.0)
    out["dx"] = d.to(dt)
    return out


def exact(case, seed):
    """The same outputs from the definitions, in 64 bits (8-bit values unrounded)."""
    st = prepare(case, seed)
    op, rows, cols = case["op"], case["rows"], case["cols"]
    parts, dgamma = [], 0.0
    step = max(1, min(rows, (1 << 23) // cols))
    gamma = None if op == "dropout" else st["gamma"].double()
    for lo in range(0, rows, step):
        sl = slice(lo, min(rows, lo + step))
        factor = 1.0
        if case["p"]:
            factor = _factors(st["rng"].cpu().numpy(), case["p"], lo, sl.stop, cols).cuda()
        o = {}
        if op == "rmsnorm_backward":
            dy, h = st["dy"][sl].double(), st["h"][sl].double()
            r = st["rstd"][sl].double()[:, None]
            n = h * r  # the normed row; d n / d h = r (1 - n n^T / cols)
            u = dy * gamma
            d = r * (u - n * (u * n).sum(1, keepdim=True) / cols)
            if st["dh"] is not None:
                d += st["dh"][sl].double()
            dgamma = dgamma + (dy * n).sum(0)
            if case["p"]:
                o["dresidual"] = d
            o["dx"] = d * factor
        else:
            h = st["x"][sl].double() * factor
            if st["res"] is not None:
                h += st["res"][sl].double()
            if op == "dropout":
                o["y"] = h
            else:
                if case["p"] or st["res"] is not None:
                    o["h"] = h
                    h = h.to(st["x"].dtype).double()
                r = (h.pow(2).sum(1) / cols + st["eps"]).pow(-0.5)
                y = h * r[:, None] * gamma
                if op == "rmsnorm":
                    o["rstd"] = r
                elif case["scale"] == "given":
                    y = (y / st["given"].double()).clamp(-E4M3_MAX, E4M3_MAX)
                elif case["scale"] == "row":
                    o["scale"] = y.abs().amax(1) / E4M3_MAX
                    y = y / o["scale"][:, None]
                else:
                    runs = y.split(128, 1)
                    o["scale"] = torch.stack([v.abs().amax(1) for v in runs], 1) / E4M3_MAX
                    y = torch.cat([v / o["scale"][:, i:i + 1] for i, v in enumerate(runs)], 1)
                o["y"] = y
        parts.append(o)
    out = {n: torch.cat([q[n] for q in parts]) for n in parts[0]}
    if op == "rmsnorm_backward":
        out["dgamma"] = dgamma
    return out["y"] if op == "dropout" else out


def _factors(rng, p, lo, hi, cols):
    """0 or 1 / (1 - t / 65536) for rows lo .. hi, by the generator's definition."""
    low = np.uint64(0xFFFFFFFF)
    half = np.uint64(32)
    seed, offset = (int(v) % 2**64 for v in rng)
    offset = (offset + SITE) % 2**64
    row, block = np.meshgrid(np.arange(lo, hi, dtype=np.uint64),
                             np.arange(-(-cols // 8), dtype=np.uint64), indexing="ij")
    ctr = [block, row, np.full_like(row, offset % 2**32), np.full_like(row, offset // 2**32)]
    for i in range(7):
        key = [np.uint64((seed % 2**32 + i * 0x9E3779B9) % 2**32),
               np.uint64((seed // 2**32 + i * 0xBB67AE85) % 2**32)]
        left, right = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(right >> half) ^ ctr[1] ^ key[0], right & low, (left >> half) ^ ctr[3] ^ key[1],
               left & low]
    bits = np.stack(ctr, 2).astype("<u4").view("<u2").reshape(hi - lo, -1)[:, :cols]
    t = _threshold(p)
    return torch.from_numpy(np.where(bits < t, 0.0, 1.0 / (1.0 - t / 65536.0)))


def work(case):
    rows, cols = case["rows"], case["cols"]
    n = rows * cols
    es = 4 if case["dtype"] == "f32" else 2
    res, drop, op = int(case["residual"]), int(case["p"] > 0), case["op"]
    if op == "dropout":  # x and the residual in, y out
        return {"bytes": n * es * (2 + res), "flops": 3 * n}
    if op == "rmsnorm":  # x and the residual in; the sum, y and rstd out
        return {"bytes": n * es * (2 + res + (res or drop)) + 4 * (cols + rows), "flops": 6 * n}
    if op == "rmsnorm_quant":  # the same with y in 8 bits and its scales
        scales = {"row": rows, "group": rows * -(-cols // 128), "given": 1}[case["scale"]]
        return {"bytes": n * (es * (1 + res + (res or drop)) + 1) + 4 * (cols + scales),
                "flops": 9 * n}
    # dy, the sum and the residual's gradient in; the gradients out
    return {"bytes": n * es * (3 + res + drop) + 4 * (2 * cols + rows), "flops": 12 * n}
