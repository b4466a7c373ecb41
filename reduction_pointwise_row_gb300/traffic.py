"""Algorithmic bytes: what each op must move between HBM and the SMs.

The count is the method's own: every input element read once, every output
element written once (the 2N bound of fused softmax, "Stax (4): GPU Codegen and
Dynamic Shapes", section 9.5), plus the small per-row vectors.  Achieved
bandwidth = these bytes / kernel time.

``naive_softmax_elements`` restates the five-kernel accounting of "CMU 15-779
Lecture 8", section 3 (amax, subtract, exp, sum, divide each reading and
writing HBM) so the tests can pin this model against the element counts that
page prints for a 1823 x 781 input.
"""
from __future__ import annotations


def naive_softmax_elements(rows: int, cols: int) -> tuple[int, int]:
    """(elements read, elements written) of the unfused 5-kernel softmax."""
    mn, m = rows * cols, rows
    reads = mn + (mn + m) + mn + mn + (mn + m)    # amax, sub, exp, sum, div
    writes = m + mn + mn + m + mn
    return reads, writes


def fused_softmax_elements(rows: int, cols: int) -> tuple[int, int]:
    return rows * cols, rows * cols


def algorithmic_bytes(op: str, rows: int, cols: int, **kw) -> int:
    if op == "relu_add_sum":          # a, b fp32 in; out fp32 [rows]
        return 2 * rows * cols * 4 + rows * 4
    if op == "relu_add_sum_bf16":     # a, b bf16 in; out fp32 [rows]
        return 2 * rows * cols * 2 + rows * 4
    if op == "sumsq":                 # x fp32 in; out fp32 [rows]
        return rows * cols * 4 + rows * 4
    if op == "softmax":               # x fp32 in; y fp32 out
        return 2 * rows * cols * 4
    if op == "softmax_offset":        # fp32 softmax, x and y out of phase: same bytes
        return 2 * rows * cols * 4
    if op == "softmax_bf16":          # x bf16 in; y bf16 out
        return 2 * rows * cols * 2
    if op == "softmax_bf16_offset":   # bf16 softmax, x and y out of phase: same bytes
        return 2 * rows * cols * 2
    if op == "layernorm":             # x bf16 in, y bf16 out, gamma/beta fp32, mean/rstd fp32
        return 2 * rows * cols * 2 + 2 * cols * 4 + 2 * rows * 4
    if op == "xent":                  # logits bf16, targets int64, loss fp32 [rows], mean fp32
        return rows * cols * 2 + rows * 8 + rows * 4 + 4
    if op == "xent_f32":              # the same with fp32 logits
        return rows * cols * 4 + rows * 8 + rows * 4 + 4
    # rows of logits (kw: dtype "bf16" or "f32", top entries a row, loss wanted, entropy's
    # gradient given); tokens and teacher indices int64, everything else a row has fp32
    logits = rows * cols * (4 if kw.get("dtype", "bf16") == "f32" else 2)
    top, loss = kw.get("top", 0), 4 * rows if kw.get("loss", True) else 0
    if op == "logprobs":              # logprob, entropy, lse and the alternatives out
        return logits + rows * (8 + 3 * 4 + 12 * top)
    if op == "logprobs_backward":     # dlogprob and dentropy in
        return 2 * logits + rows * (8 + 4 + (4 if kw.get("entropy", True) else 0))
    if op == "distill":               # teacher entries in
        return logits + rows * 12 * top + 4 * rows
    if op == "distill_backward":      # teacher entries and dloss in
        return 2 * logits + rows * (12 * top + 4) + loss
    if op == "xent_backward":         # targets and dloss in
        return 2 * logits + rows * (8 + 4) + loss
    # a residual block's row operators (kw: dtype, residual given, dropout): every matrix once
    n = rows * cols
    es = 4 if kw.get("dtype", "bf16") == "f32" else 2
    res, drop = int(kw.get("residual", False)), int(kw.get("drop", False))
    if op == "dropout":               # x and the residual in, y out
        return n * es * (2 + res)
    if op == "rmsnorm":               # the same, the sum's rounding and rstd out, gamma in
        return n * es * (2 + res + (res or drop)) + 4 * (cols + rows)
    if op == "rmsnorm_quant":         # y in 8 bits; kw scales: fp32 scales written or read
        return n * (es * (1 + res + (res or drop)) + 1) + 4 * (cols + kw.get("scales", rows))
    if op == "rmsnorm_backward":      # dy, h and dh (residual) in, the gradients out
        return n * es * (3 + res + drop) + 4 * (2 * cols + rows)
    raise ValueError(op)
