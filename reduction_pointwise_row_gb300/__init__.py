"""Fused pointwise + row-reduction kernels for GB300 (sm_103a): Python binding.

A thin ctypes layer over ``libfr.so`` (``include/fr.h``).  It only marshals
arguments -- device pointers, sizes, the current CUDA stream -- and every step of
the computation runs in the library's CUDA kernels.  PyTorch provides device
memory and streams.  There is no fallback: if the library is missing or the
device is not an sm_103 GPU the calls raise.

Functions carry the C names:

    fr_reduce_relu_add_sum(a, b, scale=2.0, form="auto")     -> out [rows] fp32
    fr_softmax(x, form="auto")                                -> y fp32
    fr_layernorm(x, gamma, beta, eps=1e-5, form="auto")       -> (y bf16, mean, rstd)
    fr_xent(logits, target, ignore_index=-100, ...)           -> dict of outputs
    fr_xent_backward(logits, target, dloss, ...)              -> dict: dlogits, loss
    fr_logprobs(logits, token, top=0, ...)                    -> dict of outputs
    fr_logprobs_backward(logits, token, dlogprob, dentropy)   -> dlogits
    fr_distill(logits, teacher_index, teacher_logit, ...)     -> loss [rows] fp32
    fr_distill_backward(logits, ..., dloss, ...)              -> dict: dlogits, loss
    fr_dropout(x, p, rng, site=0, residual=None)              -> y
    fr_rmsnorm(x, gamma, eps=1e-5, residual=None, ...)        -> dict: y, h, rstd
    fr_rmsnorm_quant(x, gamma, eps=1e-5, scale="row", ...)    -> dict: y (e4m3), scale, h
    fr_rmsnorm_backward(dy, h, gamma, rstd, dh=None, ...)     -> dict: dx, dresidual, dgamma
    fr_workspace_size(op, rows, cols, dtype, form)
    fr_check_device_error()
"""
from __future__ import annotations

import ctypes
import os

from . import buildlib as _build

__all__ = [
    "FR_OK", "FRError", "lib", "fr_version", "fr_workspace_size", "fr_last_form", "fr_auto_form",
    "fr_reduce_relu_add_sum", "fr_reduce_sumsq", "fr_softmax", "fr_softmax_host", "fr_layernorm",
    "fr_xent", "fr_xent_workspace", "fr_xent_mean_from_parts", "xent_mean_parts",
    "allreduce_mean_parts", "XENT_PARTS_OFFSET",
    "fr_reduce_relu_add_sum_split_static", "fr_check_device_error", "FORMS", "OPS",
    "EPILOGUES", "FR_TOP_MAX", "fr_logprobs", "fr_logprobs_backward", "fr_distill",
    "fr_distill_backward", "fr_xent_backward", "fr_dropout", "fr_rmsnorm", "fr_rmsnorm_quant",
    "fr_rmsnorm_backward", "SCALE_COLS", "fr_coordinate_descent", "fr_xent_get_config", "fr_xent_set_config",
    "fr_xent_tune",
]

FR_OK = 0
STATUS = {0: "FR_OK", 1: "FR_ERR_INVALID_ARG", 2: "FR_ERR_UNSUPPORTED_DTYPE",
          3: "FR_ERR_UNSUPPORTED_FORM", 4: "FR_ERR_MISALIGNED",
          5: "FR_ERR_WORKSPACE_TOO_SMALL", 6: "FR_ERR_CUDA", 7: "FR_ERR_DEVICE_DATA",
          8: "FR_ERR_NO_DEVICE"}
FORMS = {"auto": 0, "persistent": 1, "looped": 2, "split": 3}
FORM_NAMES = {v: k for k, v in FORMS.items()}
OPS = {"relu_add_sum": 0, "softmax": 1, "layernorm": 2, "xent": 3, "sumsq": 4, "logprobs": 5,
       "logprobs_backward": 6, "distill": 7, "distill_backward": 8, "xent_backward": 9,
       "rmsnorm": 10, "rmsnorm_quant": 11, "rmsnorm_backward": 12}
EPILOGUES = {"sum": 0, "sqrt": 1}
FR_TOP_MAX = 128  # most alternatives (fr_logprobs) or teacher entries (fr_distill) per row
SCALE_COLS = 128  # FR_SCALE_COLS: columns of a scale in groups (fr_rmsnorm_quant)
DTYPES = {"f32": 0, "bf16": 1}
_DTYPE_NAMES = {v: k for k, v in DTYPES.items()}

# name -> (restype, argtypes) of every symbol include/fr.h declares
_i64, _f32, _vp, _sz, _int = ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t, \
    ctypes.c_int
_i32 = ctypes.c_int32
SIGNATURES = {
    "fr_version": (_int, []),
    "fr_status_string": (ctypes.c_char_p, [_int]),
    "fr_last_form": (_int, []),
    "fr_workspace_size": (_sz, [_int, _i64, _i64, _int, _int]),
    "fr_auto_form": (_int, [_int, _int, _i64, _i64, ctypes.c_int32]),
    "fr_reduce_relu_add_sum": (_int, [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _int, _f32, _int,
                                      _vp, _sz, _vp]),
    "fr_reduce_sumsq": (_int, [_vp, _vp, _i64, _i64, _i64, _int, _int, _int, _vp, _sz, _vp]),
    "fr_softmax": (_int, [_vp, _vp, _i64, _i64, _i64, _i64, _int, _int, _vp]),
    "fr_softmax_host_workspace": (_sz, [_i64, _int, _i64]),
    "fr_softmax_host": (_int, [_vp, _vp, _i64, _i64, _int, _i64, _vp, _sz, _vp]),
    "fr_layernorm": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _f32, _int,
                            _int, _vp]),
    "fr_xent": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _int, _int, _vp,
                       _sz, _vp]),
    "fr_xent_mean_from_parts": (_int, [_vp, _vp, _vp]),
    "fr_xent_workspace_init": (_int, [_vp, _sz, _vp]),
    "fr_logprobs": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64, _i64, _int,
                           _int, _vp, _sz, _vp]),
    "fr_logprobs_backward": (_int, [_vp, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _i64,
                                    _i64, _int, _int, _vp]),
    "fr_distill": (_int, [_vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64, _i64, _f32, _int, _int,
                          _vp]),
    "fr_distill_backward": (_int, [_vp, _vp, _vp, _vp, _i64, _vp, _vp, _i32, _i64, _i64, _i64,
                                   _i64, _i64, _f32, _int, _int, _vp]),
    "fr_xent_backward": (_int, [_vp, _vp, _vp, _i64, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _int,
                                _int, _vp]),
    "fr_dropout": (_int, [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _f32, _vp, _i64, _int, _vp]),
    "fr_rmsnorm": (_int, [_vp] * 6 + [_i64] * 6 + [_f32, _f32, _vp, _i64, _int, _int, _vp]),
    "fr_rmsnorm_quant": (_int, [_vp] * 6 + [_int, _i64, _i64, _vp] + [_i64] * 6 +
                         [_f32, _f32, _vp, _i64, _int, _int, _vp]),
    "fr_rmsnorm_backward": (_int, [_vp] * 8 + [_i64] * 7 +
                            [_f32, _vp, _i64, _int, _int, _vp, _sz, _vp]),
    "fr_check_device_error": (_int, [_vp, ctypes.POINTER(ctypes.c_int32)]),
    "fr_coordinate_descent": (_int, [ctypes.c_int32, _vp, _vp, _vp, ctypes.c_double, _vp, _vp,
                                     _vp, _vp]),
    "fr_xent_get_config": (_int, [_i64, _i64, _i64, _vp]),
    "fr_xent_set_config": (_int, [_i64, _i64, _i64, _vp]),
    "fr_xent_tune": (_int, [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _int, ctypes.c_double,
                            ctypes.c_int32, _vp, _vp, _vp, _vp]),
    "fr_reduce_relu_add_sum_split_static": (_int, [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _int,
                                                   _f32, _vp]),
}


class FRError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


_lib = None


def library_path() -> str:
    return _build.LIB


def lib():
    """The loaded libfr.so (built in-tree by ``build()``; never a fallback)."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: run reduction_pointwise_row_gb300.buildlib.build() "
                              "(nvcc for sm_103a) first")
        l = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(l, name)
            f.restype, f.argtypes = res, args
        _lib = l
    return _lib


def build(force: bool = False) -> str:
    return _build.build(force=force)


def _check(status: int, where: str):
    if status != FR_OK:
        raise FRError(status, where)


_current_raw_stream = None  # device index -> cudaStream_t of its current stream
_current_device = None


def _stream(stream=None, device_index=None):
    """The raw cudaStream_t (an int) to launch on: `stream`, else the current
    stream of the current (or given) device.  The lookups are resolved once:
    a call costs two C calls, no Stream object (launch-bound shapes feel it)."""
    global _current_raw_stream, _current_device
    if stream is not None:
        return stream.cuda_stream
    if _current_raw_stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _current_raw_stream = raw if raw is not None else (  # last: it is what is tested
            lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _current_raw_stream(_current_device() if device_index is None else device_index)


def _on_current_device(*ts):
    """The library launches on the current CUDA device: refuse tensors that
    live on another one (their addresses mean nothing there)."""
    _stream()  # resolves the device lookup
    cur = _current_device()
    for t in ts:
        if t is not None and t.get_device() != cur:
            raise ValueError(f"tensor on cuda:{t.get_device()}, current device is cuda:{cur}: "
                             "call inside torch.cuda.device(...)")


def _ptr(t):
    """A tensor's device address as an int (ctypes passes it as void *), or None."""
    return t.data_ptr() if t is not None else None


def _ld(t) -> int:
    assert t.dim() == 2 and t.stride(1) == 1, "rows must be contiguous (stride(1) == 1)"
    return t.stride(0)


def fr_version() -> int:
    return lib().fr_version()


def fr_last_form() -> str:
    return FORM_NAMES[lib().fr_last_form()]


def fr_auto_form(op: str, rows: int, cols: int, dtype: str = "f32", sm_count: int = 152) -> str:
    """The form AUTO picks for this shape on a device with ``sm_count`` SMs
    (host-side; no device needed)."""
    return FORM_NAMES[lib().fr_auto_form(OPS[op], DTYPES[dtype], rows, cols, sm_count)]


def sm_count(device=None) -> int:
    """SMs of the current (or given) CUDA device."""
    import torch
    return torch.cuda.get_device_properties(
        torch.cuda.current_device() if device is None else device).multi_processor_count


def fr_workspace_size(op: str, rows: int, cols: int, dtype: str = "f32", form: str = "auto") -> int:
    return lib().fr_workspace_size(OPS[op], rows, cols, DTYPES[dtype], FORMS[form])


_WS_SIZES = {}  # (op, rows, cols, dtype, form, device index) -> bytes


def _workspace(op, rows, cols, dtype, form, device, given=None):
    import torch
    key = (op, rows, cols, dtype, form, device.index)
    n = _WS_SIZES.get(key)
    if n is None:  # depends only on the shape and the device model
        n = _WS_SIZES[key] = fr_workspace_size(op, rows, cols, dtype, form)
    if n == 0:
        return None, 0
    if given is not None:
        return given, given.numel() * given.element_size()
    return torch.empty(n, dtype=torch.uint8, device=device), n


def fr_reduce_relu_add_sum(a, b, scale: float = 2.0, form: str = "auto", out=None,
                           workspace=None, stream=None):
    """out[x] = sum_r scale * relu(a[x, r] + b[x, r]) (fp32 or bf16 in, fp32 out;
    bf16 inputs are widened exactly to fp32 before the sum)."""
    import torch
    assert a.is_cuda and b.is_cuda and a.dtype == b.dtype
    assert a.dtype in (torch.float32, torch.bfloat16)
    assert a.shape == b.shape and a.dim() == 2
    dt = "f32" if a.dtype == torch.float32 else "bf16"
    rows, cols = a.shape
    if out is None:
        out = torch.empty(rows, dtype=torch.float32, device=a.device)
    _on_current_device(a, b, out)
    ws, nws = _workspace("relu_add_sum", rows, cols, dt, form, a.device, workspace)
    _check(lib().fr_reduce_relu_add_sum(_ptr(a), _ptr(b), _ptr(out), rows, cols, _ld(a), _ld(b),
                                        DTYPES[dt], scale, FORMS[form], _ptr(ws), nws,
                                        _stream(stream)), "fr_reduce_relu_add_sum")
    return out


def fr_reduce_sumsq(x, epilogue: str = "sum", form: str = "auto", out=None, workspace=None,
                    stream=None):
    """out[x] = sum_r x[x, r]^2 (epilogue "sum") or its square root, the row L2
    norm (epilogue "sqrt"); fp32 in, fp32 out."""
    import torch
    assert x.is_cuda and x.dtype == torch.float32 and x.dim() == 2
    rows, cols = x.shape
    if out is None:
        out = torch.empty(rows, dtype=torch.float32, device=x.device)
    _on_current_device(x, out)
    ws, nws = _workspace("sumsq", rows, cols, "f32", form, x.device, workspace)
    _check(lib().fr_reduce_sumsq(_ptr(x), _ptr(out), rows, cols, _ld(x), DTYPES["f32"],
                                 EPILOGUES[epilogue], FORMS[form], _ptr(ws), nws,
                                 _stream(stream)), "fr_reduce_sumsq")
    return out


def fr_softmax(x, form: str = "auto", out=None, stream=None):
    """Row softmax of fp32 or bf16 x, y of the same dtype (returns a new tensor
    unless ``out`` is given)."""
    import torch
    assert x.is_cuda and x.dtype in (torch.float32, torch.bfloat16) and x.dim() == 2
    rows, cols = x.shape
    if out is None:
        out = torch.empty_like(x)
    assert out.dtype == x.dtype and out.shape == x.shape
    dt = DTYPES["f32"] if x.dtype == torch.float32 else DTYPES["bf16"]
    _on_current_device(x, out)
    _check(lib().fr_softmax(_ptr(x), _ptr(out), rows, cols, _ld(x), _ld(out), dt,
                            FORMS[form], _stream(stream)), "fr_softmax")
    return out


def fr_softmax_host(x_host, out=None, chunk_rows: int | None = None, workspace=None,
                    stream=None, device=None):
    """Row softmax of a page-locked host tensor (fp32 or bf16); ``out``
    (page-locked, same shape and dtype) receives y.  ``chunk_rows`` None or 0:
    the kernel reads and writes the host rows directly over the host link;
    ``chunk_rows`` >= 1: the library's chunked copy-in / kernel / copy-out
    pipeline through a device workspace.  Returns ``out``.  Ordered on
    ``stream`` (default: the current stream of ``device``) without
    synchronising."""
    import torch
    assert not x_host.is_cuda and x_host.dtype in (torch.float32, torch.bfloat16)
    assert x_host.dim() == 2 and x_host.is_contiguous()
    rows, cols = x_host.shape
    if out is None:
        out = torch.empty_like(x_host).pin_memory()
    assert out.shape == x_host.shape and out.dtype == x_host.dtype and out.is_contiguous()
    dt = DTYPES["f32"] if x_host.dtype == torch.float32 else DTYPES["bf16"]
    if chunk_rows is None:
        chunk_rows = 0
    if chunk_rows > 0 and workspace is None:
        n = lib().fr_softmax_host_workspace(cols, dt, min(chunk_rows, rows))
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    nws = 0 if workspace is None else workspace.numel()
    _check(lib().fr_softmax_host(_ptr(x_host), _ptr(out), rows, cols, dt, chunk_rows,
                                 _ptr(workspace), nws, _stream(stream)), "fr_softmax_host")
    return out


def fr_layernorm(x, gamma, beta, eps: float = 1e-5, form: str = "auto", out=None, mean=None,
                 rstd=None, stream=None):
    """LayerNorm of bf16 rows; returns (y bf16, mean fp32, rstd fp32)."""
    import torch
    assert x.is_cuda and x.dtype == torch.bfloat16 and x.dim() == 2
    rows, cols = x.shape
    assert gamma.dtype == torch.float32 and beta.dtype == torch.float32
    assert gamma.numel() == cols and beta.numel() == cols
    if out is None:
        out = torch.empty_like(x)
    if mean is None:
        mean = torch.empty(rows, dtype=torch.float32, device=x.device)
    if rstd is None:
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    _on_current_device(x, gamma, beta, out, mean, rstd)
    _check(lib().fr_layernorm(_ptr(x), _ptr(gamma), _ptr(beta), _ptr(out), _ptr(mean), _ptr(rstd),
                              rows, cols, _ld(x), _ld(out), eps, DTYPES["bf16"], FORMS[form],
                              _stream(stream)), "fr_layernorm")
    return out, mean, rstd


XENT_PARTS_OFFSET = 16  # FR_XENT_PARTS_OFFSET


def fr_xent_workspace(rows: int, cols: int, dtype: str = "bf16", device=None, stream=None):
    """A prepared cross-entropy workspace for this shape (fr_workspace_size
    bytes, prepared by fr_xent_workspace_init on ``stream``).  Every fr_xent
    call leaves it prepared; one call at a time may use it."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    n = fr_workspace_size("xent", rows, cols, dtype)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
    _check(lib().fr_xent_workspace_init(_ptr(ws), ws.numel(), _stream(stream, dev.index)),
           "fr_xent_workspace_init")
    return ws


_XENT_WS = {}  # (device, stream, bytes) -> a prepared workspace the binding reuses


def _xent_workspace_for(rows, cols, dtype, device, stream):
    """The binding's own prepared workspace for calls on this device and
    stream (calls on one stream are ordered, so they can share it)."""
    sid = _stream(stream, device.index)
    n = fr_workspace_size("xent", rows, cols, dtype)
    key = (device.index, sid)
    ws = _XENT_WS.get(key)
    if ws is None or ws.numel() < n:
        ws = fr_xent_workspace(rows, cols, dtype, device, stream)
        _XENT_WS[key] = ws
    return ws


def xent_mean_parts(workspace):
    """The two fp64 values an fr_xent call with the mean leaves in its
    workspace -- the sum of the losses it averaged and the number of rows it
    averaged -- as a view that an all-reduce can sum in place."""
    return workspace[XENT_PARTS_OFFSET:XENT_PARTS_OFFSET + 16].view(_torch().float64)


def allreduce_mean_parts(parts, group=None):
    """Sum mean parts element-wise over the ranks of ``group``
    (torch.distributed, in place): the path's one exchange step."""
    import torch.distributed as dist
    dist.all_reduce(parts, op=dist.ReduceOp.SUM, group=group)
    return parts


def fr_xent_mean_from_parts(workspace, mean=None, stream=None):
    """mean = sum / count from the (summed) parts in an fr_xent workspace."""
    import torch
    if mean is None:
        mean = torch.empty(1, dtype=torch.float32, device=workspace.device)
    _check(lib().fr_xent_mean_from_parts(_ptr(workspace), _ptr(mean), _stream(stream)),
           "fr_xent_mean_from_parts")
    return mean


_TORCH = None


def _torch():
    """torch, imported with the first call that needs it."""
    global _TORCH
    if _TORCH is None:
        import torch
        _LOGIT_DTYPES.update({torch.float32: DTYPES["f32"], torch.bfloat16: DTYPES["bf16"]})
        _TORCH = torch  # last: another thread's call that sees it finds the table filled
    return _TORCH


def _nullcontext():
    import contextlib
    return contextlib.nullcontext()


def fr_xent(logits, target, ignore_index: int = -100, want_loss: bool = True,
            want_mean: bool = True, want_target_logit: bool = False, want_argmax: bool = False,
            form: str = "auto", workspace=None, stream=None, group=None):
    """Cross entropy of bf16 or fp32 logits rows against int64 targets.

    Returns a dict with the requested outputs: ``loss`` [rows], ``mean`` [1],
    ``target_logit`` [rows], ``argmax`` [rows] (int64).  ``workspace``, when
    given, must come from fr_xent_workspace (prepared once; each call keeps
    it prepared); by default the binding keeps one per device and stream.
    With ``group`` (a
    torch.distributed group whose ranks each pass their own rows of one
    batch), ``mean`` is the mean over the whole batch: the ranks' mean parts
    are all-reduced between this rank's kernel and the finishing kernel.
    """
    import torch
    assert logits.is_cuda and logits.dtype in (torch.bfloat16, torch.float32) and logits.dim() == 2
    dt = "bf16" if logits.dtype == torch.bfloat16 else "f32"
    assert target.dtype == torch.int64 and target.is_cuda
    rows, cols = logits.shape
    assert target.numel() == rows
    dev = logits.device
    res = {}
    loss = torch.empty(rows, dtype=torch.float32, device=dev) if want_loss else None
    mean = torch.empty(1, dtype=torch.float32, device=dev) if want_mean else None
    tl = torch.empty(rows, dtype=torch.float32, device=dev) if want_target_logit else None
    am = torch.empty(rows, dtype=torch.int64, device=dev) if want_argmax else None
    _on_current_device(logits, target)
    ws, nws = (None, 0)
    if want_mean:
        ws = workspace if workspace is not None else _xent_workspace_for(rows, cols, dt, dev,
                                                                         stream)
        nws = ws.numel() * ws.element_size()
    _check(lib().fr_xent(_ptr(logits), _ptr(target), _ptr(loss), _ptr(mean), _ptr(tl), _ptr(am),
                         rows, cols, _ld(logits), ignore_index, DTYPES[dt], FORMS[form],
                         _ptr(ws), nws, _stream(stream)), "fr_xent")
    if group is not None and want_mean:
        with torch.cuda.stream(stream) if stream is not None else _nullcontext():
            allreduce_mean_parts(xent_mean_parts(ws), group)
            fr_xent_mean_from_parts(ws, mean, stream)
    for k, v in (("loss", loss), ("mean", mean), ("target_logit", tl), ("argmax", am)):
        if v is not None:
            res[k] = v
    return res


def fr_reduce_relu_add_sum_split_static(a, b, scale: float = 2.0, out=None, stream=None):
    """Split-form relu_add_sum with no workspace: the partial sums live in the
    library's fixed 64 KiB device array, so nothing is allocated for the call
    (for callers that cannot allocate device memory where they launch).  Calls
    on one device share that array: keep them ordered on one stream."""
    import torch
    assert a.is_cuda and b.is_cuda and a.dtype == torch.float32 and b.dtype == torch.float32
    assert a.shape == b.shape and a.dim() == 2
    rows, cols = a.shape
    if out is None:
        out = torch.empty(rows, dtype=torch.float32, device=a.device)
    _on_current_device(a, b, out)
    _check(lib().fr_reduce_relu_add_sum_split_static(_ptr(a), _ptr(b), _ptr(out), rows, cols,
                                                     _ld(a), _ld(b), DTYPES["f32"], scale,
                                                     _stream(stream)),
           "fr_reduce_relu_add_sum_split_static")
    return out


# ---- rows of logits: scoring, distillation, gradients ---------------------------

_LOGIT_DTYPES = {}  # torch dtype -> dtype code (filled when torch is imported)


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _logits_arg(x, name: str = "logits"):
    """(rows, cols, ld, dtype code) of a matrix of logits; refuses anything else."""
    dt = _LOGIT_DTYPES.get(x.dtype)
    if dt is None or not x.is_cuda or x.dim() != 2:
        raise ValueError(f"{name} must be a CUDA matrix of bf16 or fp32")
    rows, cols = x.shape
    ld, inner = x.stride()
    if rows < 1 or cols < 1:
        raise ValueError(f"{name} must have at least one row and one column")
    if inner != 1 and cols != 1:
        raise ValueError(f"rows of {name} must be contiguous")
    if rows == 1:  # a single row has no distance to the next one (torch may report any)
        ld = cols
    elif ld < cols:
        raise ValueError(f"rows of {name} overlap")
    return rows, cols, ld, dt


def _tokens_ptr(t, name: str, rows: int):
    """The address of int64 tokens, one per row."""
    if not t.is_cuda or t.dtype is not _TORCH.int64 or t.shape != (rows,) or \
            (rows > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous CUDA tensor of int64, one per row")
    return t.data_ptr()


def _upstream(t, name: str, rows: int) -> int:
    """The stride of an upstream gradient: fp32, one value per row or one in all."""
    if not t.is_cuda or t.dtype is not _TORCH.float32:
        raise ValueError(f"{name} must be a CUDA tensor of fp32")
    if t.numel() == 1:
        return 0
    if t.shape != (rows,):
        raise ValueError(f"{name} must hold one value, or one per row")
    return t.stride(0)


def _teacher_args(index, logit, rows: int):
    """(top, ldt) of a row's teacher entries."""
    _need(index.is_cuda and index.dtype is _TORCH.int64, "teacher_index must be int64 on CUDA")
    _need(logit.is_cuda and logit.dtype is _TORCH.float32, "teacher_logit must be fp32 on CUDA")
    _need(index.dim() == 2 and index.shape == logit.shape and index.shape[0] == rows,
          "teacher_index and teacher_logit must be [rows, top]")
    top = index.shape[1]
    _need(1 <= top <= FR_TOP_MAX, f"1 to {FR_TOP_MAX} teacher entries per row")
    (li, si), (lz, sz) = index.stride(), logit.stride()
    _need(top == 1 or si == sz == 1, "a row's teacher entries must be contiguous")
    if rows == 1:
        return top, top
    _need(li == lz, "teacher_index and teacher_logit must have the same row stride")
    _need(li >= top, "teacher rows overlap")
    return top, li


_NO_CONTEXT = _nullcontext()


def _on_stream(stream):
    """Outputs made for a call belong to the stream it runs on."""
    return _NO_CONTEXT if stream is None else _TORCH.cuda.stream(stream)


def _gradient_out(x, rows: int, cols: int, ld: int, given):
    """(dlogits, ldd): `given` after its checks, or a new matrix whose rows share
    the logits' offset within 32 bytes (a compact matrix when theirs are)."""
    if given is not None:
        _need(given.shape == x.shape and given.dtype is x.dtype,
              "dlogits must have the logits' shape and dtype")
        return given, _logits_arg(given, "dlogits")[2]
    if ld == cols:
        return _TORCH.empty((rows, cols), dtype=x.dtype, device=x.device), cols
    ldd = cols + (ld - cols) % (32 // x.element_size())
    return _TORCH.empty_strided((rows, cols), (ldd, 1), dtype=x.dtype, device=x.device), ldd


def fr_logprobs(logits, token=None, top: int = 0, ignore_index: int = -100,
                want_entropy: bool = True, want_lse: bool = True, form: str = "auto",
                workspace=None, stream=None):
    """Log probabilities of given tokens, the entropy and the top alternatives of
    each row of bf16 or fp32 logits, in one pass.

    Returns a dict: ``logprob`` [rows] (with ``token`` int64 [rows]; 0 where it
    is ``ignore_index``), ``entropy`` [rows], ``lse`` [rows], and with ``top``
    (at most min(cols, FR_TOP_MAX)) ``top_logprob`` and ``top_index`` [rows,
    top], the largest first, ties by the lower index.  All fp32 but the int64
    ``top_index``.  ``workspace``: fr_workspace_size("logprobs", ...) bytes, by
    default allocated for the call."""
    torch = _TORCH or _torch()
    rows, cols, ld, dt = _logits_arg(logits)
    if not 0 <= top <= min(cols, FR_TOP_MAX):
        raise ValueError(f"top must be 0 to min(cols, {FR_TOP_MAX})")
    _on_current_device(logits, token, workspace)
    _need(workspace is None or workspace.is_contiguous(), "workspace must be contiguous")
    dev, f32 = logits.device, torch.float32
    res = {}
    p_token = p_lp = p_ent = p_lse = p_tl = p_ti = p_ws = None
    nws = 0
    with _on_stream(stream):
        if token is not None:
            p_token = _tokens_ptr(token, "token", rows)
            t = res["logprob"] = torch.empty(rows, dtype=f32, device=dev)
            p_lp = t.data_ptr()
        if want_entropy:
            t = res["entropy"] = torch.empty(rows, dtype=f32, device=dev)
            p_ent = t.data_ptr()
        if want_lse:
            t = res["lse"] = torch.empty(rows, dtype=f32, device=dev)
            p_lse = t.data_ptr()
        if top > 0:
            t = res["top_logprob"] = torch.empty((rows, top), dtype=f32, device=dev)
            p_tl = t.data_ptr()
            t = res["top_index"] = torch.empty((rows, top), dtype=torch.int64, device=dev)
            p_ti = t.data_ptr()
            ws, nws = _workspace("logprobs", rows, cols, _DTYPE_NAMES[dt], form, dev, workspace)
            p_ws = _ptr(ws)
        _need(bool(res), "no output requested")
    status = lib().fr_logprobs(logits.data_ptr(), p_token, p_lp, p_ent, p_lse, p_tl, p_ti, top,
                               rows, cols, ld, ignore_index, dt, FORMS[form], p_ws, nws,
                               _stream(stream))
    _check(status, "fr_logprobs")
    return res


def fr_logprobs_backward(logits, token=None, dlogprob=None, dentropy=None,
                         ignore_index: int = -100, dlogits=None, form: str = "auto",
                         stream=None):
    """The gradient of fr_logprobs' ``logprob`` and ``entropy`` with respect to the
    logits, from fp32 upstream gradients with one value per row or one in all
    (either may be None).  ``dlogits`` may be ``logits`` (in place)."""
    _TORCH or _torch()
    rows, cols, ld, dt = _logits_arg(logits)
    _need(dlogprob is not None or dentropy is not None, "no upstream gradient given")
    _need(dlogprob is None or token is not None, "dlogprob needs the tokens")
    p_token = None if token is None else _tokens_ptr(token, "token", rows)
    gs = 0 if dlogprob is None else _upstream(dlogprob, "dlogprob", rows)
    hs = 0 if dentropy is None else _upstream(dentropy, "dentropy", rows)
    with _on_stream(stream):
        dlogits, ldd = _gradient_out(logits, rows, cols, ld, dlogits)
    _on_current_device(logits, token, dlogprob, dentropy, dlogits)
    _check(lib().fr_logprobs_backward(logits.data_ptr(), p_token, _ptr(dlogprob), gs,
                                      _ptr(dentropy), hs, dlogits.data_ptr(), rows, cols, ld, ldd,
                                      ignore_index, dt, FORMS[form], _stream(stream)),
           "fr_logprobs_backward")
    return dlogits


def fr_distill(logits, teacher_index, teacher_logit, temperature: float = 1.0,
               form: str = "auto", stream=None):
    """The distillation loss [rows] (fp32) of bf16 or fp32 logits against a teacher's
    top logits: temperature^2 KL(softmax(teacher_logit / T) || softmax(logits /
    T)) over the entries of ``teacher_index`` (int64 [rows, top], negative:
    padding) and ``teacher_logit`` (fp32 [rows, top]; log probabilities serve)."""
    torch = _TORCH or _torch()
    rows, cols, ld, dt = _logits_arg(logits)
    top, ldt = _teacher_args(teacher_index, teacher_logit, rows)
    _on_current_device(logits, teacher_index, teacher_logit)
    with _on_stream(stream):
        loss = torch.empty(rows, dtype=torch.float32, device=logits.device)
    _check(lib().fr_distill(logits.data_ptr(), teacher_index.data_ptr(), teacher_logit.data_ptr(),
                            loss.data_ptr(), top, rows, cols, ld, ldt, temperature, dt,
                            FORMS[form], _stream(stream)), "fr_distill")
    return loss


def fr_distill_backward(logits, teacher_index, teacher_logit, dloss, temperature: float = 1.0,
                        want_loss: bool = True, dlogits=None, form: str = "auto", stream=None):
    """The gradient of fr_distill's loss and, with ``want_loss``, the loss of the
    same pass: a training step in one call.  Returns a dict: ``dlogits`` and
    ``loss``.  ``dloss`` holds one fp32 value per row or one in all; ``dlogits``
    may be ``logits`` (in place)."""
    torch = _TORCH or _torch()
    rows, cols, ld, dt = _logits_arg(logits)
    top, ldt = _teacher_args(teacher_index, teacher_logit, rows)
    gs = _upstream(dloss, "dloss", rows)
    p_loss = None
    with _on_stream(stream):
        dlogits, ldd = _gradient_out(logits, rows, cols, ld, dlogits)
        res = {"dlogits": dlogits}
        if want_loss:
            t = res["loss"] = torch.empty(rows, dtype=torch.float32, device=logits.device)
            p_loss = t.data_ptr()
    _on_current_device(logits, teacher_index, teacher_logit, dloss, dlogits)
    _check(lib().fr_distill_backward(logits.data_ptr(), teacher_index.data_ptr(),
                                     teacher_logit.data_ptr(), dloss.data_ptr(), gs, p_loss,
                                     dlogits.data_ptr(), top, rows, cols, ld, ldd, ldt,
                                     temperature, dt, FORMS[form], _stream(stream)),
           "fr_distill_backward")
    return res


def fr_xent_backward(logits, target, dloss, ignore_index: int = -100, want_loss: bool = True,
                     dlogits=None, form: str = "auto", stream=None):
    """The gradient of fr_xent's per-row loss and, with ``want_loss``, that loss from
    the same pass.  Returns a dict: ``dlogits`` and ``loss``.  ``dloss`` holds one
    fp32 value per row or one in all (1 / counted rows gives the mean's
    gradient); ``dlogits`` may be ``logits`` (in place)."""
    torch = _TORCH or _torch()
    rows, cols, ld, dt = _logits_arg(logits)
    p_target = _tokens_ptr(target, "target", rows)
    gs = _upstream(dloss, "dloss", rows)
    p_loss = None
    with _on_stream(stream):
        dlogits, ldd = _gradient_out(logits, rows, cols, ld, dlogits)
        res = {"dlogits": dlogits}
        if want_loss:
            t = res["loss"] = torch.empty(rows, dtype=torch.float32, device=logits.device)
            p_loss = t.data_ptr()
    _on_current_device(logits, target, dloss, dlogits)
    _check(lib().fr_xent_backward(logits.data_ptr(), p_target, dloss.data_ptr(), gs, p_loss,
                                  dlogits.data_ptr(), rows, cols, ld, ldd, ignore_index, dt,
                                  FORMS[form], _stream(stream)), "fr_xent_backward")
    return res


# ---- a residual block's row operators: dropout, root-mean-square norm ------------
#
# Small calls are bound by the host, so a call looks at each tensor once, mostly inline,
# and enters a context only for a given `stream` (fr_rmsnorm of one row: 15.4 us, 18.9 before; 3.7
# of it the library's call, about 2 each output's allocation).


def _device_of(x) -> int:
    """x's device, which has to be the current one (the library launches there)."""
    dev = x.get_device()
    if _current_raw_stream is None:
        _stream()  # resolves the lookups; this one is published last
    if dev != _current_device():
        _on_current_device(x)
    return dev


def _like(t, x, ld: int, dev: int, name: str) -> int:
    """The row stride of a matrix that has to have x's shape, dtype and device."""
    if t.dtype is x.dtype and t.shape == x.shape and t.is_cuda:
        if t.get_device() != dev:
            _on_current_device(t)
        return ld if t.stride() == x.stride() else _logits_arg(t, name)[2]
    raise ValueError(f"{name} must be on CUDA and have the first matrix's shape and dtype")


def _vector_ptr(t, n: int, dev: int, name: str) -> int:
    """The address of n contiguous fp32 values."""
    if t.dtype is _TORCH.float32 and t.shape == (n,) and t.is_cuda and t.is_contiguous():
        if t.get_device() != dev:
            _on_current_device(t)
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous CUDA tensor of {n} fp32 values")


def _rng_ptr(p: float, rng, site: int, dev: int):
    """The address of a call's {seed, offset}; None without dropout."""
    if not -2**63 <= site < 2**63:
        raise ValueError("site must fit 64 bits")
    if 0.0 <= p <= 2.0**-150:  # the library takes p in fp32: 0 there
        return None
    if not 0.0 < p <= 1.0:
        raise ValueError("p must be 0 to 1")
    if rng is None or not rng.is_cuda or rng.dtype is not _TORCH.int64 or rng.shape != (2,) or \
            not rng.is_contiguous():
        raise ValueError("rng must be a contiguous CUDA tensor of two int64: seed and offset")
    if rng.get_device() != dev:
        _on_current_device(rng)
    return rng.data_ptr()


def _matrix_out(x, rows: int, cols: int, ld: int):
    """(matrix, row stride): a new one of x's shape and dtype whose rows share x's offset
    within 8 elements (a compact matrix when x is one)."""
    if ld == cols:
        if x.is_contiguous():
            return _TORCH.empty_like(x), cols
        return _TORCH.empty((rows, cols), dtype=x.dtype, device=x.device), cols
    ldo = cols + (ld - cols) % 8
    return _TORCH.empty_strided((rows, cols), (ldo, 1), dtype=x.dtype, device=x.device), ldo


def _with_stream(call, stream, *args):
    """The call with `stream` as the current one: what it makes belongs to it."""
    _torch()
    with _TORCH.cuda.stream(stream):
        return call(*args)


def fr_dropout(x, p: float, rng, site: int = 0, residual=None, out=None, stream=None):
    """residual + dropout(x) (residual None: dropout(x)) of bf16 or fp32 rows.  The
    mask is drawn from ``rng``, an int64 CUDA tensor {seed, offset}, ``site`` and the
    element's row and column, and never stored: the gradient of x is fr_dropout of
    y's gradient with the same rng, site and p.  offset + site is one number: advance the
    offset between steps by at least the number of sites, or one place's mask is
    another's of the step before.  ``out`` may be x or residual; a new matrix's rows lie as
    x's do within 8 elements (compact where x is)."""
    if stream is not None:
        return _with_stream(fr_dropout, stream, x, p, rng, site, residual, out)
    _TORCH or _torch()
    rows, cols, ld, dt = _logits_arg(x, "x")
    dev = _device_of(x)
    p_rng = _rng_ptr(p, rng, site, dev)
    ldr = 0 if residual is None else _like(residual, x, ld, dev, "residual")
    if out is None:
        out, ldo = _matrix_out(x, rows, cols, ld)
    else:
        ldo = _like(out, x, ld, dev, "out")
    status = lib().fr_dropout(x.data_ptr(), None if residual is None else residual.data_ptr(),
                              out.data_ptr(), rows, cols, ld, ldr, ldo, p, p_rng, site, dt,
                              _current_raw_stream(dev))
    if status != FR_OK:
        raise FRError(status, "fr_dropout")
    return out


def fr_rmsnorm(x, gamma, eps: float = 1e-5, residual=None, p: float = 0.0, rng=None, site: int = 0,
               want_rstd: bool = True, form: str = "auto", out=None, h=None, rstd=None, stream=None):
    """Root-mean-square norm of bf16 or fp32 rows after the residual's addition:
    h = residual + dropout(x), y = h / sqrt(mean(h^2) + eps) * gamma (fp32).

    Returns a dict: ``y``; ``h`` where there is a residual or dropout (else the
    norm's input is x); ``rstd`` [rows] fp32 for the backward pass.  ``out`` and
    ``h`` may be x or residual.  Dropout as in fr_dropout."""
    if stream is not None:
        return _with_stream(fr_rmsnorm, stream, x, gamma, eps, residual, p, rng, site, want_rstd, form,
                            out, h, rstd)
    _TORCH or _torch()
    rows, cols, ld, dt = _logits_arg(x, "x")
    dev = _device_of(x)
    p_gamma = _vector_ptr(gamma, cols, dev, "gamma")
    p_rng = _rng_ptr(p, rng, site, dev)
    ldr = ldh = 0
    ldy = cols
    p_res = p_h = p_rstd = None
    if residual is not None:
        ldr = _like(residual, x, ld, dev, "residual")
        p_res = residual.data_ptr()
    if out is None:
        out, ldy = _matrix_out(x, rows, cols, ld)
    else:
        ldy = _like(out, x, ld, dev, "out")
    res = {"y": out}
    if p_res is not None or p_rng is not None:
        if h is None:
            h, ldh = _matrix_out(x, rows, cols, ld)
        else:
            ldh = _like(h, x, ld, dev, "h")
        p_h = h.data_ptr()
        res["h"] = h
    elif h is not None:
        raise ValueError("h without a residual or dropout: the norm's input is x itself")
    if rstd is not None:
        p_rstd = _vector_ptr(rstd, rows, dev, "rstd")
        res["rstd"] = rstd
    elif want_rstd:
        rstd = res["rstd"] = _TORCH.empty(rows, dtype=_TORCH.float32, device=x.device)
        p_rstd = rstd.data_ptr()
    status = lib().fr_rmsnorm(x.data_ptr(), p_res, p_gamma, p_h, out.data_ptr(), p_rstd, rows, cols, ld,
                              ldr, ldh, ldy, eps, p, p_rng, site, dt, FORMS[form],
                              _current_raw_stream(dev))
    if status != FR_OK:
        raise FRError(status, "fr_rmsnorm")
    return res


def _scale_strides(t, rows: int, groups: int, dev: int):
    """(row stride, group stride) of scales [rows] (groups 0) or [rows, groups]."""
    if not t.is_cuda or t.dtype is not _TORCH.float32 or \
            t.shape != ((rows, groups) if groups else (rows,)):
        raise ValueError("scale_out must be a CUDA tensor of fp32, one per row (or group)")
    if t.get_device() != dev:
        _on_current_device(t)
    if not groups:
        return t.stride(0) if rows > 1 else 1, 1
    sr, sc = t.stride()
    if rows == 1:  # a dimension of one element has no stride that counts
        sr = groups if sc == 1 else 1
    if groups == 1:
        sc = 1 if sr != 1 else rows
    return sr, sc


def fr_rmsnorm_quant(x, gamma, eps: float = 1e-5, scale="row", residual=None, p: float = 0.0,
                     rng=None, site: int = 0, want_rstd: bool = False, form: str = "auto", out=None,
                     scale_out=None, h=None, rstd=None, stream=None):
    """fr_rmsnorm with y in 8 bits (torch.float8_e4m3fn), y * scale being the norm.

    ``scale``: "row" (one scale a row, max |y| / 448), "group" (one per 128 columns of
    a row) or a CUDA tensor of one fp32 value, which is used as it is (below 2^-126 as
    2^-126).  Returns a
    dict: ``y``; ``scale`` ([rows], or [rows, groups], where it is not given); ``h``
    and ``rstd`` as fr_rmsnorm.  ``scale_out`` takes the scales in a tensor of the
    caller's, groups in either order ([rows, groups] with one stride of 1)."""
    if stream is not None:
        return _with_stream(fr_rmsnorm_quant, stream, x, gamma, eps, scale, residual, p, rng, site,
                            want_rstd, form, out, scale_out, h, rstd)
    torch = _TORCH or _torch()
    rows, cols, ld, dt = _logits_arg(x, "x")
    dev = _device_of(x)
    p_gamma = _vector_ptr(gamma, cols, dev, "gamma")
    p_rng = _rng_ptr(p, rng, site, dev)
    ldr = ldh = 0
    ldy = cols
    p_res = p_h = p_rstd = None
    if residual is not None:
        ldr = _like(residual, x, ld, dev, "residual")
        p_res = residual.data_ptr()
    if out is None:
        ldy = cols + (ld - cols) % 8
        out = torch.empty_strided((rows, cols), (ldy, 1), dtype=torch.float8_e4m3fn, device=x.device)
    else:
        if not out.is_cuda or out.dtype is not torch.float8_e4m3fn or out.shape != x.shape or \
                (out.stride(1) != 1 and cols != 1):
            raise ValueError("out must be a CUDA matrix of float8_e4m3fn, x's shape")
        if out.get_device() != dev:
            _on_current_device(out)
        ldy = cols if rows == 1 else out.stride(0)
    res = {"y": out}
    sr = sc = 1
    if isinstance(scale, str):
        if scale == "row":
            mode, groups = 0, 0
        elif scale == "group":
            mode, groups = 1, -(-cols // SCALE_COLS)
            sr = groups
        else:
            raise ValueError('scale must be "row", "group" or a tensor of one fp32 value')
        if scale_out is None:
            scale_out = torch.empty((rows, groups) if groups else rows, dtype=torch.float32, device=x.device)
        else:
            sr, sc = _scale_strides(scale_out, rows, groups, dev)
        p_scale = scale_out.data_ptr()
        res["scale"] = scale_out
    else:
        mode = 2
        _need(scale_out is None, "scale_out with a given scale")
        _need(isinstance(scale, torch.Tensor) and scale.is_cuda and scale.dtype is torch.float32 and
              scale.numel() == 1, 'scale must be "row", "group" or a CUDA tensor of one fp32 value')
        if scale.get_device() != dev:
            _on_current_device(scale)
        p_scale = scale.data_ptr()
    if p_res is not None or p_rng is not None:
        if h is None:
            h, ldh = _matrix_out(x, rows, cols, ld)
        else:
            ldh = _like(h, x, ld, dev, "h")
        p_h = h.data_ptr()
        res["h"] = h
    elif h is not None:
        raise ValueError("h without a residual or dropout: the norm's input is x itself")
    if rstd is not None:
        p_rstd = _vector_ptr(rstd, rows, dev, "rstd")
        res["rstd"] = rstd
    elif want_rstd:
        rstd = res["rstd"] = _TORCH.empty(rows, dtype=_TORCH.float32, device=x.device)
        p_rstd = rstd.data_ptr()
    status = lib().fr_rmsnorm_quant(x.data_ptr(), p_res, p_gamma, p_h, out.data_ptr(), p_scale, mode, sr,
                                    sc, p_rstd, rows, cols, ld, ldr, ldh, ldy, eps, p, p_rng, site, dt,
                                    FORMS[form], _current_raw_stream(dev))
    if status != FR_OK:
        raise FRError(status, "fr_rmsnorm_quant")
    return res


def fr_rmsnorm_backward(dy, h, gamma, rstd, dh=None, p: float = 0.0, rng=None, site: int = 0,
                        want_dgamma: bool = True, want_dresidual: bool = True, form: str = "auto",
                        dx=None, dresidual=None, dgamma=None, workspace=None, stream=None):
    """The gradient of fr_rmsnorm from ``dy`` and, with ``dh``, the gradient that
    reaches h by the residual's path.  ``h`` and ``rstd`` are the forward pass's (h: x
    where it had neither residual nor dropout).

    Returns a dict: ``dx``, the gradient of x; ``dgamma`` [cols] fp32; and with
    dropout (p, rng and site as in the forward pass) ``dresidual``, the gradient of
    the residual, which without dropout is dx.  ``dx`` and ``dresidual`` may be given,
    also as dy, h or dh.  ``workspace``: fr_workspace_size("rmsnorm_backward", ...)
    bytes, by default allocated for the call."""
    if stream is not None:
        return _with_stream(fr_rmsnorm_backward, stream, dy, h, gamma, rstd, dh, p, rng, site,
                            want_dgamma, want_dresidual, form, dx, dresidual, dgamma, workspace)
    _TORCH or _torch()
    rows, cols, ld, dt = _logits_arg(dy, "dy")
    dev = _device_of(dy)
    ldh = _like(h, dy, ld, dev, "h")
    p_gamma = _vector_ptr(gamma, cols, dev, "gamma")
    p_rstd = _vector_ptr(rstd, rows, dev, "rstd")
    p_rng = _rng_ptr(p, rng, site, dev)
    lddh = lddr = 0
    lddx = cols
    p_dh = p_dr = p_dg = None
    if dh is not None:
        lddh = _like(dh, dy, ld, dev, "dh")
        p_dh = dh.data_ptr()
    if workspace is not None:
        if not (workspace.is_cuda and workspace.is_contiguous()):
            raise ValueError("workspace must be contiguous CUDA memory")
        if workspace.get_device() != dev:
            _on_current_device(workspace)
    if dx is None:
        dx, lddx = _matrix_out(dy, rows, cols, ld)
    else:
        lddx = _like(dx, dy, ld, dev, "dx")
    res = {"dx": dx}
    if p_rng is None:
        _need(dresidual is None, "dresidual without dropout is dx")
    else:
        if dresidual is not None:
            lddr = _like(dresidual, dy, ld, dev, "dresidual")
        elif want_dresidual:
            dresidual, lddr = _matrix_out(dy, rows, cols, ld)
        if dresidual is not None:
            p_dr = dresidual.data_ptr()
            res["dresidual"] = dresidual
    if dgamma is not None:
        p_dg = _vector_ptr(dgamma, cols, dev, "dgamma")
        res["dgamma"] = dgamma
    elif want_dgamma:
        dgamma = res["dgamma"] = _TORCH.empty(cols, dtype=_TORCH.float32, device=dy.device)
        p_dg = dgamma.data_ptr()
    ws, nws = _workspace("rmsnorm_backward", rows, cols, _DTYPE_NAMES[dt], form, dy.device, workspace)
    status = lib().fr_rmsnorm_backward(dy.data_ptr(), h.data_ptr(), p_gamma, p_rstd, p_dh, dx.data_ptr(),
                                       p_dr, p_dg, rows, cols, ld, ldh, lddh, lddx, lddr, p, p_rng, site,
                                       dt, FORMS[form], _ptr(ws), nws, _current_raw_stream(dev))
    if status != FR_OK:
        raise FRError(status, "fr_rmsnorm_backward")
    return res


# ---- launch configurations ----------------------------------------------------

COST_FN = ctypes.CFUNCTYPE(ctypes.c_double, ctypes.POINTER(ctypes.c_int32), ctypes.c_void_p)


class XentConfig(ctypes.Structure):
    _fields_ = [("threads", ctypes.c_int32), ("vectors", ctypes.c_int32),
                ("stages", ctypes.c_int32), ("ctas_per_sm", ctypes.c_int32)]

    def as_tuple(self):
        return (self.threads, self.vectors, self.stages, self.ctas_per_sm)


def fr_coordinate_descent(lo, hi, start, eps: float, cost):
    """Coordinate descent (Algorithm 9.2) over log2 parameters in the box
    [lo, hi] from ``start``; ``cost(tuple)`` returns a time (inf: cannot run).
    Returns (result, acceptances, evaluations)."""
    p = len(start)
    arr = ctypes.c_int32 * p
    c_lo, c_hi, c = arr(*lo), arr(*hi), arr(*start)
    fn = COST_FN(lambda q, _ctx: float(cost(tuple(q[i] for i in range(p)))))
    acc, ev = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(lib().fr_coordinate_descent(p, ctypes.byref(c_lo), ctypes.byref(c_hi),
                                       ctypes.byref(c), eps, ctypes.cast(fn, ctypes.c_void_p),
                                       None, ctypes.byref(acc), ctypes.byref(ev)),
           "fr_coordinate_descent")
    return tuple(c), acc.value, ev.value


def fr_xent_get_config(rows: int, cols: int, ld: int | None = None) -> tuple:
    out = XentConfig()
    _check(lib().fr_xent_get_config(rows, cols, cols if ld is None else ld, ctypes.byref(out)),
           "fr_xent_get_config")
    return out.as_tuple()


def fr_xent_set_config(rows: int, cols: int, cfg, ld: int | None = None):
    """Records (threads, vectors, stages, ctas_per_sm) for this shape; None forgets."""
    ptr = None if cfg is None else ctypes.byref(XentConfig(*cfg))
    _check(lib().fr_xent_set_config(rows, cols, cols if ld is None else ld, ptr),
           "fr_xent_set_config")


def fr_xent_tune(logits, target, ignore_index: int = -100, eps: float = 0.02, reps: int = 5,
                 loss=None, stream=None) -> dict:
    """Algorithm 9.1 + 9.2 on the caller's data; records and returns the chosen
    configuration with the number of configurations timed and its median ms."""
    import torch
    assert logits.is_cuda and logits.dtype == torch.bfloat16 and logits.dim() == 2
    rows, cols = logits.shape
    out, ev, ms = XentConfig(), ctypes.c_int32(0), ctypes.c_float(0)
    _check(lib().fr_xent_tune(_ptr(logits), _ptr(target), _ptr(loss), rows, cols, _ld(logits),
                              ignore_index, DTYPES["bf16"], eps, reps, _stream(stream),
                              ctypes.byref(out), ctypes.byref(ev), ctypes.byref(ms)),
           "fr_xent_tune")
    return {"config": out.as_tuple(), "evaluations": ev.value, "ms": ms.value}


def fr_check_device_error(stream=None) -> int:
    """Synchronises the stream; returns and clears the device error code (0 = none)."""
    code = ctypes.c_int32(0)
    st = lib().fr_check_device_error(_stream(stream), ctypes.byref(code))
    if st not in (FR_OK, 7):
        raise FRError(st, "fr_check_device_error")
    return code.value
