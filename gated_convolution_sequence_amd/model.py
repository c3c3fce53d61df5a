"""The operators between the layers of a sequence model and its weights.

A thin binding of the C ABI in ``include/hyena_model.h`` (libhyena_model.so),
in the manner of the package's other calls: it checks and marshals arguments,
every step of the computation runs in the library's HIP kernels, and there is
no fallback.  What a call writes into tensors that it was given raises their version, as
torch's own in-place operations do, so that a graph that has saved one of them refuses its backward.

norm_fwd, norm_bwd      layer norm and root-mean-square norm of rows (Norm: autograd)
xent_fwd, xent_bwd      softmax cross entropy of a readout, no logits kept (LinearXent: autograd)
grad_norm, adamw_step   the norm of all gradients and an AdamW step over a list of tensors
"""
from __future__ import annotations

import array
import ctypes
import functools
import operator
import os
from typing import Optional, Sequence, Tuple, Union

import torch
from torch.autograd.graph import increment_version

from . import HyenaError  # the package imports this module last
from ._autograd import first_order
from .layer import _code, _contiguous, _like, _on_stream, _pick, _ptr, _rows_of, _shared_stride, _workspace, _ws_args

_PKG = os.path.dirname(os.path.abspath(__file__))
MODEL_LIB_PATH = os.path.join(_PKG, "libhyena_model.so")

NORMS = {"layer": 0, "rms": 1}

# Every function include/hyena_model.h declares.
MODEL_EXPORTS = ("hyena_norm_fwd", "hyena_norm_bwd", "hyena_norm_workspace", "hyena_xent_fwd", "hyena_xent_bwd",
                 "hyena_xent_workspace", "hyena_adamw_step", "hyena_grad_norm", "hyena_grad_norm_workspace",
                 "hyena_model_strerror")

_lib = None


class ModelError(HyenaError):
    """A status of the library other than HYENA_OK, with this library's text for it."""

    def __init__(self, status: int, where: str):
        self.status = status
        RuntimeError.__init__(self, "%s: %s (%d)" % (where, model_strerror(status), status))


def model_lib() -> ctypes.CDLL:
    """The loaded library of these operators; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(MODEL_LIB_PATH):
            raise RuntimeError(
                "libhyena_model.so is not built (expected at %s); run "
                "`python -c 'import __graft_entry__ as g; g.build()'`" % MODEL_LIB_PATH)
        L = ctypes.CDLL(MODEL_LIB_PATH)
        vp, i64, ci, cf, cd = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_double
        out = ctypes.POINTER(i64)
        for name, args in (
                ("hyena_norm_fwd", [vp] * 3 + [i64] * 4 + [ci, cf] + [vp] * 3 + [ci, vp]),
                ("hyena_norm_bwd", [vp] * 5 + [i64] * 5 + [ci] + [vp] * 4 + [i64, ci, vp]),
                ("hyena_norm_workspace", [i64, i64, ci, out]),
                ("hyena_xent_fwd", [vp] * 4 + [i64] * 4 + [vp] * 3 + [i64, ci, vp]),
                ("hyena_xent_bwd", [vp] * 6 + [i64] * 5 + [vp] * 4 + [i64, ci, vp]),
                ("hyena_xent_workspace", [i64, i64, i64, ci, ci, out]),
                ("hyena_adamw_step", [vp, i64] + [cd] * 5 + [i64] * 2 + [vp] * 4 + [ci, ci, vp]),
                ("hyena_grad_norm", [vp, i64, cd] + [vp] * 3 + [i64, ci, vp]),
                ("hyena_grad_norm_workspace", [i64, i64, out])):
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ci
        L.hyena_model_strerror.argtypes = [ci]
        L.hyena_model_strerror.restype = ctypes.c_char_p
        _lib = L
    return _lib


def model_strerror(status: int) -> str:
    return model_lib().hyena_model_strerror(int(status)).decode()


def _call(name: str, dev: torch.device, *args) -> None:
    """name(*args, current stream) on dev; raises ModelError for a status other than HYENA_OK."""
    fn = getattr(_lib or model_lib(), name)
    handle = torch._C._cuda_getCurrentRawStream(dev.index)
    if dev.index == torch._C._cuda_getDevice():
        st = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, handle)
    if st != 0:
        raise ModelError(st, name)


def _bytes(name: str, *args) -> int:
    n = ctypes.c_int64()
    st = getattr(model_lib(), name)(*args, ctypes.byref(n))
    if st != 0:
        raise ModelError(st, name)
    return n.value


# ---- norm over a row's channels ----------------------------------------------------

@functools.lru_cache(maxsize=1024)
def norm_workspace_bytes(M: int, D: int, dtype: int = 0) -> int:
    """Workspace bytes norm_bwd needs for M rows of D channels."""
    return _bytes("hyena_norm_workspace", M, D, dtype)


@_on_stream
def norm_fwd(x: torch.Tensor, w: Optional[torch.Tensor] = None, b: Optional[torch.Tensor] = None,
             kind: str = "layer", eps: float = 1e-5, save_stats: bool = False, out: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None):
    """(y, mean, rstd): y = (x - mean) rstd w + b over the last dimension.

    x: [..., D] (bf16 or fp32), rows at one stride; w, b: [D] of x's type (None:
    1 and 0).  kind: "layer" (mean and deviation) or "rms" (mean is 0).  mean
    and rstd ([...] fp32) are returned with ``save_stats`` (mean only for "layer"),
    else None.
    """
    code = _code(x)
    kcode = _pick(NORMS, kind, "kind")
    dev, dt = x.device, x.dtype
    if x.dim() < 1:
        raise ValueError("x must be [..., D]")
    D = x.shape[-1]
    M = x.numel() // D if D else _rows_of(x)
    ldx = ldy = D
    if not x.is_contiguous():
        ldx = _shared_stride((x,), ("x",), D)
    _contiguous(w, "w", (D,), dt, dev)
    _contiguous(b, "b", (D,), dt, dev)
    given = out
    if out is None:
        out = torch.empty(x.shape, dtype=dt, device=dev)
    else:
        _like(out, "out", x.shape, dt, dev)
        ldy = _shared_stride((out,), ("out",), D)
    mean = rstd = None
    if save_stats:
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
        if kcode == 0:
            mean = torch.empty_like(rstd)
    _call("hyena_norm_fwd", dev, x.data_ptr(), _ptr(w), _ptr(b), M, D, ldx, ldy, kcode, eps, out.data_ptr(),
          _ptr(mean), _ptr(rstd), code)
    if given is not None:
        increment_version(given)
    return out, mean, rstd


@_on_stream
def norm_bwd(x: torch.Tensor, w: Optional[torch.Tensor], dy: torch.Tensor, mean: Optional[torch.Tensor],
             rstd: torch.Tensor, kind: str = "layer", need_dx: bool = True, need_dw: bool = True,
             need_db: bool = True, dx: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None):
    """Gradients (dx, dw, db) of norm_fwd for upstream dy ([..., D], rows at one stride).

    mean (None for "rms") and rstd are what norm_fwd returned with
    save_stats.  Parts not requested are None; dw also where w is None.  ``dx`` may be
    given to be written to.
    """
    code = _code(x)
    kcode = _pick(NORMS, kind, "kind")
    dev, dt = x.device, x.dtype
    if x.dim() < 1:
        raise ValueError("x must be [..., D]")
    D = x.shape[-1]
    M = x.numel() // D if D else _rows_of(x)
    ldx = lddy = lddx = D
    if not x.is_contiguous():
        ldx = _shared_stride((x,), ("x",), D)
    _contiguous(w, "w", (D,), dt, dev)
    _like(dy, "dy", x.shape, dt, dev)
    if not dy.is_contiguous():
        lddy = _shared_stride((dy,), ("dy",), D)
    if (mean is None) != (kcode == 1):
        raise ValueError("mean is what norm_fwd saved: a tensor for kind 'layer', None for 'rms'")
    _contiguous(mean, "mean", x.shape[:-1], torch.float32, dev)
    _contiguous(rstd, "rstd", x.shape[:-1], torch.float32, dev)
    given = dx if need_dx else None
    if not need_dx:
        dx = None
    elif dx is None:
        dx = torch.empty(x.shape, dtype=dt, device=dev)
    else:
        _like(dx, "dx", x.shape, dt, dev)
        lddx = _shared_stride((dx,), ("dx",), D)
    dw = torch.empty((D,), dtype=dt, device=dev) if need_dw and w is not None else None
    db = torch.empty((D,), dtype=dt, device=dev) if need_db else None
    if dx is None and dw is None and db is None:
        return None, None, None
    ws = _workspace(norm_workspace_bytes(M, D, code), workspace, dev)
    _call("hyena_norm_bwd", dev, x.data_ptr(), _ptr(w), dy.data_ptr(), _ptr(mean), rstd.data_ptr(), M, D, ldx, lddy,
          lddx, kcode, _ptr(dx), _ptr(dw), _ptr(db), *_ws_args(ws), code)
    if given is not None:
        increment_version(given)
    return dx, dw, db


class Norm(torch.autograd.Function):
    """Autograd wrapper: y = Norm.apply(x, w, b, kind, eps); w and b may be None.  No second derivatives: they raise."""

    @staticmethod
    def forward(ctx, x, w=None, b=None, kind="layer", eps=1e-5):
        y, mean, rstd = norm_fwd(x, w, b, kind=kind, eps=eps, save_stats=True)
        ctx.save_for_backward(x, w, mean, rstd, b)
        ctx.kind = kind
        return y

    @staticmethod
    @first_order
    def backward(ctx, dy):
        x, w, mean, rstd, _ = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = norm_bwd(x, w, dy.contiguous(), mean, rstd, kind=ctx.kind, need_dx=need[0],
                              need_dw=len(need) > 1 and need[1], need_db=len(need) > 2 and need[2])
        grads = (dx, dw, db, None, None)
        return tuple(t if n else None for t, n in zip(grads, need))  # as many as apply was given


# ---- softmax cross entropy of a readout ---------------------------------------------

@functools.lru_cache(maxsize=1024)
def xent_workspace_bytes(M: int, K: int, V: int, dtype: int = 0, backward: bool = False) -> int:
    """Workspace bytes xent_fwd (or xent_bwd) needs."""
    return _bytes("hyena_xent_workspace", M, K, V, dtype, int(backward))


def _xent_inputs(x, w, target, bias):
    code = _code(x)
    dev, dt = x.device, x.dtype
    if x.dim() < 1 or w.dim() != 2 or x.shape[-1] != w.shape[1]:
        raise ValueError("x must be [..., K] and w [V, K]")
    V, K = w.shape
    ldx = K if x.is_contiguous() else _shared_stride((x,), ("x",), K)
    _contiguous(w, "w", (V, K), dt, dev)
    _contiguous(bias, "bias", (V,), dt, dev)
    _contiguous(target, "target", x.shape[:-1], torch.int64, dev)
    return code, _rows_of(x), K, V, ldx


@_on_stream
def xent_fwd(x: torch.Tensor, w: torch.Tensor, target: torch.Tensor, bias: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(loss, lse) of each row: lse = log sum_v exp(z_v), loss = lse - z_target for z = x w^T + bias.

    x: [..., K], rows at one stride; w: [V, K]; bias: [V]; all of one type.
    target: int64 [...]; a row whose target is outside [0, V) (-100, say) has none:
    its loss and lse are 0.  loss, lse: fp32 [...].  The logits are not kept.
    """
    code, M, K, V, ldx = _xent_inputs(x, w, target, bias)
    dev = x.device
    loss = torch.empty(target.shape, dtype=torch.float32, device=dev)
    lse = torch.empty_like(loss)
    ws = _workspace(xent_workspace_bytes(M, K, V, code), workspace, dev)
    _call("hyena_xent_fwd", dev, x.data_ptr(), w.data_ptr(), _ptr(bias), target.data_ptr(), M, K, V, ldx,
          loss.data_ptr(), lse.data_ptr(), *_ws_args(ws), code)
    return loss, lse


@_on_stream
def xent_bwd(x: torch.Tensor, w: torch.Tensor, target: torch.Tensor, lse: torch.Tensor, dloss: torch.Tensor,
             bias: Optional[torch.Tensor] = None, need_dx: bool = True, need_dw: bool = True, need_db: bool = True,
             dx: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None):
    """Gradients (dx, dw, db) of xent_fwd's loss for upstream dloss (fp32, one a row).

    lse is the forward's.  Rows without a target get a gradient of 0 and add
    nothing to dw and db, whatever their x holds.  Parts not requested are None; db also
    where bias is None.  ``dx`` may be given to be written to.  In bf16
    softmax - [target], for dw with dloss in it or in x, is rounded to bf16 before its products, as the
    matrix cores take it; db sums unrounded values.
    """
    code, M, K, V, ldx = _xent_inputs(x, w, target, bias)
    dev, dt = x.device, x.dtype
    _contiguous(lse, "lse", target.shape, torch.float32, dev)
    _contiguous(dloss, "dloss", target.shape, torch.float32, dev)
    lddx = K
    given = dx if need_dx else None
    if not need_dx:
        dx = None
    elif dx is None:
        dx = torch.empty(x.shape, dtype=dt, device=dev)
    else:
        _like(dx, "dx", x.shape, dt, dev)
        lddx = _shared_stride((dx,), ("dx",), K)
    dw = torch.empty((V, K), dtype=dt, device=dev) if need_dw else None
    db = torch.empty((V,), dtype=dt, device=dev) if need_db and bias is not None else None
    if dx is None and dw is None and db is None:
        return None, None, None
    ws = _workspace(xent_workspace_bytes(M, K, V, code, backward=True), workspace, dev)
    _call("hyena_xent_bwd", dev, x.data_ptr(), w.data_ptr(), _ptr(bias), target.data_ptr(), lse.data_ptr(),
          dloss.data_ptr(), M, K, V, ldx, lddx, _ptr(dx), _ptr(dw), _ptr(db), *_ws_args(ws), code)
    if given is not None:
        increment_version(given)
    return dx, dw, db


class LinearXent(torch.autograd.Function):
    """Autograd wrapper: loss = LinearXent.apply(x, w, target, bias), fp32, one a row; bias may be None.

    No second derivatives: they raise.
    """

    @staticmethod
    def forward(ctx, x, w, target, bias=None):
        loss, lse = xent_fwd(x, w, target, bias=bias)
        ctx.save_for_backward(x, w, target, lse, bias)
        return loss

    @staticmethod
    @first_order
    def backward(ctx, dloss):
        x, w, target, lse, bias = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = xent_bwd(x, w, target, lse, dloss.contiguous(), bias=bias, need_dx=need[0], need_dw=need[1],
                              need_db=len(need) > 3 and need[3])
        grads = (dx, dw, None, db)
        return tuple(t if n else None for t, n in zip(grads, need))  # as many as apply was given


# ---- AdamW over many tensors ------------------------------------------------------------

_shape, _dtype = operator.attrgetter("shape"), operator.attrgetter("dtype")


class _Tensor(ctypes.Structure):
    """hyena_tensor of hyena_model.h: eight words of 64 bits."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scale",
                                               "exp_avg_sq_scale", "master")] + [("numel", ctypes.c_int64)]


def _column(table: list, at: int, ts, name: str, shapes, dtype, dev) -> None:
    """The addresses of ts into every eighth word of ``table`` from ``at`` on.

    ts has a tensor for each of ``shapes``, contiguous, ``dtype`` and on ``dev``.
    """
    if len(ts) != len(shapes):
        raise ValueError("%s has %d tensors, expected %d" % (name, len(ts), len(shapes)))
    if (list(map(_shape, ts)) != shapes or not all(map(torch.Tensor.is_contiguous, ts))
            or any(d is not dtype for d in map(_dtype, ts)) or set(map(torch.Tensor.get_device, ts)) != {dev.index}):
        raise ValueError("every tensor of %s must be contiguous %s on %s, shaped as its like" % (name, dtype, dev))
    table[at::8] = map(torch.Tensor.data_ptr, ts)


def _scalar(t: Optional[torch.Tensor], name: str, dtype, dev) -> None:
    if t is not None and (t.dtype is not dtype or t.device != dev or t.numel() != 1):
        raise ValueError("%s must be one %s on %s" % (name, dtype, dev))


@functools.lru_cache(maxsize=1024)
def grad_norm_workspace_bytes(n: int, numel: int) -> int:
    """Workspace bytes grad_norm needs for n tensors of ``numel`` elements together."""
    return _bytes("hyena_grad_norm_workspace", n, numel)


@_on_stream
def grad_norm(grads: Sequence[torch.Tensor], max_norm: Optional[float] = None,
              workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """(norm, scale) of a list of gradients (all bf16 or all fp32, contiguous), each one fp32 on their device.

    norm is the root of the sum of all squares (summed in 64 bits); scale, with ``max_norm``, is
    min(1, max_norm / norm) for adamw_step's ``grad_scale``, NaN where the norm is not finite, else None.
    """
    if len(grads) == 0:
        raise ValueError("grads is empty")
    code = _code(grads[0])
    dev = grads[0].device
    table = [0] * (8 * len(grads))
    _column(table, 1, grads, "grads", [g.shape for g in grads], grads[0].dtype, dev)
    table[7::8] = sizes = [g.numel() for g in grads]
    words = array.array("q", table)
    norm = torch.empty((), dtype=torch.float32, device=dev)
    scale = None if max_norm is None else torch.empty((), dtype=torch.float32, device=dev)
    ws = _workspace(grad_norm_workspace_bytes(len(grads), sum(sizes)), workspace, dev)
    _call("hyena_grad_norm", dev, words.buffer_info()[0], len(grads), 0.0 if max_norm is None else max_norm,
          norm.data_ptr(), _ptr(scale), *_ws_args(ws), code)
    return norm, scale


STATE_BLOCK = 256  # elements that share a scale where the moments have 8 bits


@_on_stream
def adamw_step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], exp_avgs: Sequence[torch.Tensor],
               exp_avg_sqs: Sequence[torch.Tensor], step: Union[int, torch.Tensor],
               lr: Union[float, torch.Tensor], betas: Tuple[float, float] = (0.9, 0.999), eps: float = 1e-8,
               weight_decay: float = 0.0, masters: Optional[Sequence[torch.Tensor]] = None,
               grad_scale: Optional[torch.Tensor] = None,
               exp_avg_scales: Optional[Sequence[torch.Tensor]] = None,
               exp_avg_sq_scales: Optional[Sequence[torch.Tensor]] = None,
               seed: Union[int, torch.Tensor, None] = None, stream: Optional[torch.cuda.Stream] = None) -> None:
    """One AdamW step over lists of tensors, in place, in a launch for every 48 of them.

    params, grads: all bf16 or all fp32; masters (None, or the fp32 values of which params are the roundings, and
    which then take the step); exp_avgs, exp_avg_sqs: the moments m and v in fp32, or m and sqrt(v) in
    float8_e4m3fn with exp_avg_scales and exp_avg_sq_scales, an fp32 vector for each parameter with one scale for
    every 256 elements (codes and scales of zeros to begin with; rounding is random, by ``seed``, which should
    differ from step to step; None: the step's number, or what the step's tensor holds).  All contiguous, shaped as
    params.  step counts from 1.  lr, step and seed may be one-element tensors on the device (fp32, int64, int64), which a captured step reads anew in each replay.
    grad_scale: one fp32 on the device that multiplies the gradients; where it is not finite the step is skipped.
    Without masters, a bf16 parameter loses moves below half a unit of its last place.
    """
    if len(params) == 0:
        raise ValueError("params is empty")
    code = _code(params[0])
    dev, dt = params[0].device, params[0].dtype
    bits = 8 if len(exp_avgs) and exp_avgs[0].dtype is torch.float8_e4m3fn else 32
    held, fp32 = (torch.float8_e4m3fn if bits == 8 else torch.float32), torch.float32
    table = [0] * (8 * len(params))
    shapes = [p.shape for p in params]
    _column(table, 0, params, "params", shapes, dt, dev)
    _column(table, 1, grads, "grads", shapes, dt, dev)
    _column(table, 2, exp_avgs, "exp_avgs", shapes, held, dev)
    _column(table, 3, exp_avg_sqs, "exp_avg_sqs", shapes, held, dev)
    if masters is not None:
        _column(table, 6, masters, "masters", shapes, fp32, dev)
    table[7::8] = sizes = [p.numel() for p in params]
    if bits == 8:
        blocks = [(-(-n // STATE_BLOCK),) for n in sizes]
        _column(table, 4, () if exp_avg_scales is None else exp_avg_scales, "exp_avg_scales", blocks, fp32, dev)
        _column(table, 5, () if exp_avg_sq_scales is None else exp_avg_sq_scales, "exp_avg_sq_scales", blocks, fp32, dev)
    elif exp_avg_scales is not None or exp_avg_sq_scales is not None:
        raise ValueError("scales belong to moments in float8_e4m3fn")
    if seed is None:
        seed = step
    given = [t if isinstance(t, torch.Tensor) else None for t in (lr, step, seed)]
    for t, name, kind in zip((*given, grad_scale), ("lr", "step", "seed", "grad_scale"),
                             (torch.float32, torch.int64, torch.int64, torch.float32)):
        _scalar(t, name, kind, dev)
    words = array.array("q", table)
    number = [x if t is None else zero for x, t, zero in zip((lr, step, seed), given, (0.0, 1, 0))]
    _call("hyena_adamw_step", dev, words.buffer_info()[0], len(params), number[0], betas[0], betas[1], eps,
          weight_decay, number[1], number[2], *(_ptr(t) for t in given), _ptr(grad_scale), bits, code)
    written = [*params, *exp_avgs, *exp_avg_sqs]
    for ts in (masters, exp_avg_scales, exp_avg_sq_scales):
        if ts is not None:
            written.extend(ts)
    increment_version(written)
