"""Measured cases of the row operators over a vocabulary's logits: log
probabilities with entropy and top alternatives, distillation from a teacher's
top logits, cross entropy's gradient, and the backward passes.

``listed()`` and ``draw()`` give the cases, ``prepare()`` makes a case's inputs
on the GPU from a seed, ``run()`` computes one pass -- in elementary torch
operations where ``own`` is false, through the library's calls where it is true
-- and ``exact()`` gives the same outputs in 64 bits.
"""
import math

import torch

own = False

OPS = ("logprobs", "logprobs_backward", "distill", "distill_backward", "xent_backward")
IGNORE = -100


def _case(name, op, rows, cols, dtype="bf16", ld=0, pad=0, top=0, temperature=1.0, entropy=True,
          loss=True):
    """ld: distance between row starts (0: cols); pad: trailing columns masked
    to -inf (a vocabulary padded to a round size); top: alternatives or teacher
    entries per row; entropy: logprobs_backward with the entropy's gradient;
    loss: a backward pass that also gives the loss of its rows."""
    c = dict(op=op, rows=rows, cols=cols, dtype=dtype, ld=max(ld, cols), pad=pad, top=top,
             temperature=temperature, entropy=entropy, loss=loss)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decoded token of one request, with the alternatives an API returns: latency
        _case("logprobs_decode_1", "logprobs", 1, 50257, top=20),
        # a decode step of a batch, fp32 logits over a larger vocabulary of odd size
        _case("logprobs_batch_61_f32", "logprobs", 61, 65537, "f32", top=5),
        # scoring a prompt batch: every position's token, entropy and alternatives
        _case("logprobs_score_8192", "logprobs", 8192, 50257, top=20),
        # a teacher's pass for distillation: many alternatives a row, padded vocabulary
        _case("logprobs_teacher_2048", "logprobs", 2048, 131072, pad=100, top=64),
        # policy-gradient training with an entropy bonus
        _case("logprobs_bwd_2048", "logprobs_backward", 2048, 50257),
        # supervised log-likelihood training in fp32 on an odd vocabulary
        _case("logprobs_bwd_511_f32", "logprobs_backward", 511, 32001, "f32", entropy=False),
        # a distillation training step: loss and gradient, the logits a view of a padded matrix
        _case("distill_step_4096", "distill_backward", 4096, 50257, ld=50304, top=64,
              temperature=2.0),
        # the same for a small micro-batch in fp32
        _case("distill_step_96_f32", "distill_backward", 96, 32000, "f32", top=20),
        # evaluation of the distillation loss alone
        _case("distill_eval_1024", "distill", 1024, 50257, top=32, temperature=2.0),
        # the backward pass of an autograd step whose forward pass gave the loss
        _case("distill_bwd_1022", "distill_backward", 1022, 65537, top=100, temperature=3.0,
              loss=False),
        # a cross-entropy training step: loss and gradient
        _case("xent_bwd_4096", "xent_backward", 4096, 50257),
        # a fine-tuning head over a small label set
        _case("xent_bwd_33_f32", "xent_backward", 33, 1000, "f32"),
    ]


def draw(rng):
    op = rng.choice(OPS)
    dtype = rng.choice(("bf16", "bf16", "f32"))
    cols = int(math.exp(rng.uniform(math.log(200), math.log(200000))))
    most = 2.0e8 / cols / (2 if dtype == "f32" else 1)
    rows = max(1, int(math.exp(rng.uniform(0.0, math.log(min(8192.0, most))))))
    pad = rng.choice((0, 0, rng.randint(1, 100)))
    ld = cols + rng.choice((0, 0, rng.randint(1, 64)))
    top = 0
    if op.startswith("distill"):
        top = rng.randint(1, 128)
    elif op == "logprobs":
        top = rng.choice((0, rng.randint(1, 20), rng.randint(21, 100)))
    top = min(top, (cols - pad) // 2)
    return _case("", op, rows, cols, dtype, ld, pad, top,
                 rng.choice((1.0, 1.5, 2.0, 4.0)) if op.startswith("distill") else 1.0,
                 rng.random() < 0.5, rng.random() < 0.5)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    rows, cols, ld, k, op = (case[n] for n in ("rows", "cols", "ld", "top", "op"))

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    def randint(n, *shape):
        return torch.randint(0, n, shape, generator=g, device="cuda")

    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    buf = torch.empty(rows, ld, dtype=dt, device="cuda")
    buf.normal_(0.0, 3.0, generator=g)
    x = buf[:, :cols]
    live = cols - case["pad"]
    token = randint(live, rows)
    x.scatter_add_(1, token[:, None], (6.0 * rand(rows, 1)).to(dt))  # a likely token, as trained models give
    st = dict(case, x=x, token=torch.where(rand(rows) < 0.05, IGNORE, token))
    if op.startswith("distill"):
        # distinct indexes, values falling from the top; a varying number of entries is live
        step = live // k
        idx = torch.arange(k, device="cuda") * step + randint(step, rows, k)
        val = 14.0 - torch.cumsum(-torch.log1p(-rand(rows, k)), 1) * (8.0 / k)
        x.scatter_add_(1, idx, (0.5 * val).to(dt))
        keep = torch.arange(k, device="cuda") < 1 + (k * (0.5 + rand(rows, 1))).long()
        st["t_index"] = torch.where(keep, idx, -1)
        st["t_logit"] = val
    if case["pad"]:
        x[:, live:] = -math.inf
    if op == "logprobs_backward":
        st["dlogprob"] = torch.randn(rows, generator=g, device="cuda") / rows
        st["dentropy"] = -0.01 * rand(rows) / rows if case["entropy"] else None
    if op == "distill_backward":
        st["dloss"] = rand(rows) / rows
    if op == "xent_backward":
        st["dloss"] = (1.0 / (st["token"] != IGNORE).sum().clamp(min=1)).float().reshape(1)
    return st


def _own(st):
    import reduction_pointwise_row_gb300 as fr

    op, x = st["op"], st["x"]
    if op == "logprobs":
        r = fr.fr_logprobs(x, st["token"], top=st["top"], ignore_index=IGNORE)
        return {n: r[n] for n in _logprobs_names(st)}
    if op == "logprobs_backward":
        return {"dlogits": fr.fr_logprobs_backward(x, st["token"], dlogprob=st["dlogprob"],
                                                   dentropy=st["dentropy"], ignore_index=IGNORE)}
    if op == "distill":
        return {"loss": fr.fr_distill(x, st["t_index"], st["t_logit"],
                                      temperature=st["temperature"])}
    if op == "distill_backward":
        r = fr.fr_distill_backward(x, st["t_index"], st["t_logit"], st["dloss"],
                                   temperature=st["temperature"], want_loss=st["loss"])
    else:
        r = fr.fr_xent_backward(x, st["token"], st["dloss"], ignore_index=IGNORE,
                                want_loss=st["loss"])
    return {n: r[n] for n in (["loss"] if st["loss"] else []) + ["dlogits"]}


def _logprobs_names(st):
    return ["logprob", "entropy", "lse"] + (["top_logprob", "top_index"] if st["top"] else [])


def _softmax_parts(z):
    m = z.amax(1, keepdim=True)
    d = z - m
    e = torch.exp(d)
    s = e.sum(1, keepdim=True)
    return m, d, e, s


def _teacher(st):
    """The teacher's probabilities and their logarithms; padding entries give 0."""
    live = st["t_index"] >= 0
    z = torch.where(live, st["t_logit"] / st["temperature"], -math.inf)
    m, d, e, s = _softmax_parts(z)
    return e / s, torch.where(live, d - torch.log(s), 0.0), st["t_index"].clamp(min=0)


def run(st):
    if own:
        return _own(st)
    op, dt = st["op"], st["x"].dtype
    x = st["x"].float()
    m, d, e, s = _softmax_parts(x / st["temperature"] if op.startswith("distill") else x)
    out = {}
    if op.startswith("logprobs"):
        gone = st["token"] == IGNORE
        at = st["token"].clamp(min=0)[:, None]
        entropy = torch.log(s) - (e * d.clamp(min=-1e30)).sum(1, keepdim=True) / s
    if op == "logprobs":
        out["logprob"] = torch.where(gone, 0.0, (d.gather(1, at) - torch.log(s))[:, 0])
        out["entropy"] = entropy[:, 0]
        out["lse"] = (m + torch.log(s))[:, 0]
        if st["top"]:
            v, i = torch.sort(x, dim=1, descending=True, stable=True)
            out["top_logprob"] = (v[:, :st["top"]] - m) - torch.log(s)
            out["top_index"] = i[:, :st["top"]].contiguous()
    elif op == "logprobs_backward":
        g = torch.where(gone, 0.0, st["dlogprob"])[:, None]
        p = e / s
        grad = p * -g
        if st["entropy"]:
            logp = d.clamp(min=-1e30) - torch.log(s)
            grad -= st["dentropy"][:, None] * p * (logp + entropy)
        grad.scatter_add_(1, at, g)
        out["dlogits"] = grad.to(dt)
    elif op.startswith("distill"):
        q, logq, at = _teacher(st)
        if op == "distill" or st["loss"]:
            logp = d.gather(1, at) - torch.log(s)
            out["loss"] = st["temperature"] ** 2 * torch.where(q > 0, q * (logq - logp), 0.0).sum(1)
        if op == "distill_backward":
            p = (e / s).scatter_add_(1, at, -q)
            out["dlogits"] = (p * (st["dloss"][:, None] * st["temperature"])).to(dt)
    else:
        gone = st["token"] == IGNORE
        at = st["token"].clamp(min=0)[:, None]
        loss = torch.log(s) - d.gather(1, at)
        grad = (e / s).scatter_add_(1, at, -torch.ones_like(loss))
        grad *= torch.where(gone, 0.0, st["dloss"])[:, None]
        if st["loss"]:
            out["loss"] = torch.where(gone, 0.0, loss[:, 0])
        out["dlogits"] = grad.to(dt)
    return out


def exact(case, seed):
    """The same outputs from the definitions, in 64 bits (None for indexes)."""
    st = prepare(case, seed)
    op, temp, rows = case["op"], case["temperature"], case["rows"]
    parts = []
    for lo in range(0, rows, 512):
        sl = slice(lo, min(rows, lo + 512))
        z = st["x"][sl].double() / temp
        t = st["token"][sl]
        r = torch.arange(z.shape[0], device="cuda")
        hit = t != IGNORE
        lse = torch.logsumexp(z, 1)
        logp = z - lse[:, None]
        p = logp.exp()
        o = {}
        if op == "logprobs":
            o["logprob"] = torch.where(hit, logp[r, t.clamp(min=0)], 0.0)
            o["entropy"] = -torch.nan_to_num(p * logp, nan=0.0).sum(1)
            o["lse"] = lse
            if case["top"]:
                o["top_logprob"] = torch.topk(logp, case["top"], 1).values
                o["top_index"] = None
        elif op == "logprobs_backward":
            onehot = torch.zeros_like(p)
            onehot[r[hit], t[hit]] = 1.0
            g = (st["dlogprob"][sl].double() * hit)[:, None]
            dx = g * (onehot - p)
            if case["entropy"]:
                plogp = torch.nan_to_num(p * logp, nan=0.0)
                ent = -plogp.sum(1, keepdim=True)
                dx -= st["dentropy"][sl].double()[:, None] * (plogp + p * ent)
            o["dlogits"] = dx
        elif op == "xent_backward":
            if case["loss"]:
                o["loss"] = torch.where(hit, -logp[r, t.clamp(min=0)], 0.0)
            p[r[hit], t[hit]] -= 1.0
            o["dlogits"] = p * (st["dloss"].double() * hit)[:, None]
        else:
            live = st["t_index"][sl] >= 0
            q = torch.softmax(torch.where(live, st["t_logit"][sl].double() / temp, -math.inf), 1)
            at = st["t_index"][sl].clamp(min=0)
            if op == "distill" or case["loss"]:
                term = torch.xlogy(q, q) - q * torch.where(live, logp.gather(1, at), 0.0)
                o["loss"] = temp * temp * term.sum(1)
            if op == "distill_backward":
                dense = torch.zeros_like(p).scatter_add_(1, at, q)
                o["dlogits"] = temp * st["dloss"][sl].double()[:, None] * (p - dense)
        parts.append(o)
    return {n: None if parts[0][n] is None else torch.cat([q[n] for q in parts])
            for n in parts[0]}


def work(case):
    rows, cols, k = case["rows"], case["cols"], case["top"]
    n = rows * cols
    es = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op == "logprobs":  # logits and tokens in; three floats and the alternatives out
        return {"bytes": n * es + rows * (8 + 12 + 12 * k), "flops": 6 * n}
    if op == "logprobs_backward":
        return {"bytes": 2 * n * es + rows * (16 if case["entropy"] else 12),
                "flops": (11 if case["entropy"] else 8) * n}
    if op == "distill":
        return {"bytes": n * es + rows * (12 * k + 4), "flops": 4 * n}
    loss = 4 if case["loss"] else 0
    if op == "distill_backward":
        return {"bytes": 2 * n * es + rows * (12 * k + 4 + loss), "flops": 8 * n}
    return {"bytes": 2 * n * es + rows * (8 + loss) + 4, "flops": 8 * n}
