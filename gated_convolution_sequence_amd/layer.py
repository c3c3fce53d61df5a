"""The operators around the gated convolution in a sequence layer.

A thin binding of the C ABI in ``include/hyena_layer.h`` (libhyena_layer.so),
in the manner of the package's convolution calls: it checks and marshals
arguments, every step of the computation runs in the library's HIP kernels,
and there is no fallback.

scan_fwd, scan_bwd, scan_step   gated linear recurrence along time (GatedScan: autograd)
linear_fwd, linear_bwd          matrix product with bias, activation and residual (LinearAct: autograd)
conv_step, conv_cache_fill      the gated convolution for one token at a time
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Sequence

import torch

from . import HyenaError  # the package imports this module last
from ._autograd import first_order

_PKG = os.path.dirname(os.path.abspath(__file__))
LAYER_LIB_PATH = os.path.join(_PKG, "libhyena_layer.so")

STATE_ROWS = 64  # rows between the states scan_fwd saves
GATES = {"sigmoid": 0, "log": 1}
ACTS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3, "sigmoid": 4}

# Every symbol include/hyena_layer.h declares.
LAYER_EXPORTS = ("hyena_scan_fwd", "hyena_scan_bwd", "hyena_scan_workspace", "hyena_scan_step",
                 "hyena_conv_step", "hyena_conv_cache_fill", "hyena_linear_fwd", "hyena_linear_bwd",
                 "hyena_linear_workspace", "hyena_layer_strerror")

_DTYPE_CODES = {torch.bfloat16: 0, torch.float32: 1}
_lib = None


class LayerError(HyenaError):
    """A status of the library other than HYENA_OK, with this library's text for it."""

    def __init__(self, status: int, where: str):
        self.status = status
        RuntimeError.__init__(self, "%s: %s (%d)" % (where, layer_strerror(status), status))


def layer_lib() -> ctypes.CDLL:
    """The loaded library of these operators; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LAYER_LIB_PATH):
            raise RuntimeError(
                "libhyena_layer.so is not built (expected at %s); run "
                "`python -c 'import __graft_entry__ as g; g.build()'`" % LAYER_LIB_PATH)
        L = ctypes.CDLL(LAYER_LIB_PATH)
        vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        out = ctypes.POINTER(i64)
        for name, args in (
                ("hyena_scan_fwd", [vp] * 4 + [i64] * 4 + [ci] + [vp] * 5 + [i64, ci, vp]),
                ("hyena_scan_bwd", [vp] * 7 + [i64] * 5 + [ci] + [vp] * 6 + [i64, ci, vp]),
                ("hyena_scan_workspace", [i64, i64, i64, ci, out]),
                ("hyena_scan_step", [vp] * 4 + [i64] * 3 + [ci, vp, vp, i64, vp, vp, ci, vp]),
                ("hyena_conv_step", [vp] * 4 + [i64] * 5 + [vp, i64, i64, vp, vp, vp, ci, vp]),
                ("hyena_conv_cache_fill", [vp] * 2 + [i64] * 4 + [vp, i64, i64, vp, vp, ci, vp]),
                ("hyena_linear_fwd", [vp] * 4 + [i64] * 6 + [ci, vp, vp, vp, i64, ci, vp]),
                ("hyena_linear_bwd", [vp] * 4 + [i64] * 6 + [ci] + [vp] * 4 + [i64, ci, vp]),
                ("hyena_linear_workspace", [i64, i64, i64, ci, ci, ci, out])):
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ci
        L.hyena_layer_strerror.argtypes = [ci]
        L.hyena_layer_strerror.restype = ctypes.c_char_p
        _lib = L
    return _lib


def layer_strerror(status: int) -> str:
    return layer_lib().hyena_layer_strerror(int(status)).decode()


# ---- argument checks ----------------------------------------------------------

def _code(t: torch.Tensor) -> int:
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError("tensors must be bfloat16 or float32, got %s" % t.dtype)
    if not t.is_cuda:
        raise ValueError("tensors must be on the GPU")
    return code


def _pick(table: dict, key: str, what: str) -> int:
    code = table.get(key)
    if code is None:
        raise ValueError("%s must be one of %s, got %r" % (what, ", ".join(sorted(table)), key))
    return code


def _row_stride(t: torch.Tensor, name: str) -> Optional[int]:
    """Elements from one row of t ([..., n]) to the next; None where it has at most one row."""
    shape, stride = t.shape, t.stride()
    if t.numel() == 0:
        return None
    if shape[-1] > 1 and stride[-1] != 1:
        raise ValueError("%s must have contiguous rows" % name)
    ld, rows = None, 1
    for n, s in zip(shape[-2::-1], stride[-2::-1]):
        if n == 1:
            continue
        if ld is None:
            ld = s
        elif s != ld * rows:
            raise ValueError("%s must have its rows at one stride" % name)
        rows *= n
    if ld is not None and ld < shape[-1]:
        raise ValueError("%s has overlapping rows" % name)
    return ld


def _shared_stride(ts, names, n: int) -> int:
    """The row stride that all of ts, of one shape, share (n where none has a second row)."""
    ld = _row_stride(ts[0], names[0])
    first = ts[0].stride()
    for t, name in zip(ts[1:], names[1:]):
        if t.stride() != first and _row_stride(t, name) != ld:
            raise ValueError("%s must have one row stride" % ", ".join(names))
    return n if ld is None else ld


def _like(t: torch.Tensor, name: str, shape, dtype, dev) -> None:
    if t.shape != shape or t.dtype is not dtype or t.device != dev:
        raise ValueError("%s must be %s %s on %s" % (name, tuple(shape), dtype, dev))


def _rows_like(ts, names, shape, dtype, dev) -> int:
    """The one row stride of ts, which must all be ``shape``, ``dtype`` and on ``dev``."""
    first = ts[0].stride()
    for t in ts:
        if t.shape != shape or t.dtype is not dtype or t.device != dev or t.stride() != first:
            break
    else:  # alike, as they nearly always are
        if len(shape) == 2 and first[1] == 1 and first[0] >= shape[1]:
            return first[0] if shape[0] > 1 else shape[1]
    for t, name in zip(ts, names):
        _like(t, name, shape, dtype, dev)
    return _shared_stride(ts, names, shape[-1])


def _contiguous(t: Optional[torch.Tensor], name: str, shape, dtype, dev) -> None:
    if t is not None:
        _like(t, name, shape, dtype, dev)
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _on_stream(fn):
    """Runs fn with its ``stream`` as the current one.

    What fn allocates (outputs, workspaces it does not return) then belongs to
    that stream, so that the allocator hands none of it on before its work there is done.
    """
    @functools.wraps(fn)
    def run(*args, stream: Optional[torch.cuda.Stream] = None, **kwargs):
        if stream is None:
            return fn(*args, **kwargs)
        with torch.cuda.stream(stream):
            return fn(*args, **kwargs)
    return run


def _call(name: str, dev: torch.device, *args) -> None:
    """name(*args, current stream) on dev; raises LayerError for a status other than HYENA_OK."""
    fn = getattr(_lib or layer_lib(), name)
    # the current stream's handle, without the Stream object torch.cuda.current_stream makes
    handle = torch._C._cuda_getCurrentRawStream(dev.index)
    if dev.index == torch._C._cuda_getDevice():
        st = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, handle)
    if st != 0:
        raise LayerError(st, name)


def _workspace(need: int, given: Optional[torch.Tensor], dev) -> Optional[torch.Tensor]:
    if given is None:
        return torch.empty(need, dtype=torch.uint8, device=dev) if need > 0 else None
    if given.device != dev or not given.is_contiguous() or given.numel() * given.element_size() < need:
        raise ValueError("workspace must hold %d bytes on %s" % (need, dev))
    return given


def _ws_args(ws: Optional[torch.Tensor]):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())


# ---- gated linear recurrence ------------------------------------------------------

@functools.lru_cache(maxsize=1024)
def scan_workspace_bytes(B: int, L: int, D: int, dtype: int = 0) -> int:
    """Workspace bytes scan_fwd and scan_bwd need."""
    n = ctypes.c_int64()
    st = layer_lib().hyena_scan_workspace(B, L, D, dtype, ctypes.byref(n))
    if st != 0:
        raise LayerError(st, "hyena_scan_workspace")
    return n.value


def _scan_inputs(ts, names):
    q = ts[0]
    code = _code(q)
    if q.dim() != 3:
        raise ValueError("q, k, v, g must be [B, L, D]")
    return code, _rows_like(ts, names, q.shape, q.dtype, q.device)


@_on_stream
def scan_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, gate: str = "sigmoid",
             s0: Optional[torch.Tensor] = None, save_states: bool = False, out: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """(y, s_last, states) of s_t = a_t s_{t-1} + k_t v_t, y_t = q_t s_t along dim 1.

    q, k, v, g: [B, L, D] (bf16 or fp32, all alike), rows contiguous and at one
    row stride for the four: separate contiguous tensors or column slices of
    one [B, L, 4 D] projection.  gate: "sigmoid" (a = sigmoid(g)) or "log"
    (a = exp(g), also above 1; exp(g) and the states have to fit fp32); g = -inf
    starts afresh from that row.  s0: [B, D] fp32 state before row 0 (None:
    zero).  s_last: [B, D] fp32.  states: with ``save_states`` the fp32 states
    before rows 0, 64, 128, ... that scan_bwd takes, else None.  ``workspace``
    (uint8) is allocated here if not given.
    """
    code, ld = _scan_inputs((q, k, v, g), ("q", "k", "v", "g"))
    gcode = _pick(GATES, gate, "gate")
    dev = q.device
    B, L, D = q.shape
    _contiguous(s0, "s0", (B, D), torch.float32, dev)
    if out is None:
        out = torch.empty((B, L, D), dtype=q.dtype, device=dev)
    else:
        _contiguous(out, "out", (B, L, D), q.dtype, dev)
    s_last = torch.empty((B, D), dtype=torch.float32, device=dev)
    states = None
    if save_states:
        states = torch.empty((B, -(-L // STATE_ROWS), D), dtype=torch.float32, device=dev)
    ws = _workspace(scan_workspace_bytes(B, L, D, code), workspace, dev)
    _call("hyena_scan_fwd", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), B, L, D, ld, gcode,
          _ptr(s0), out.data_ptr(), s_last.data_ptr(), _ptr(states), *_ws_args(ws), code)
    return out, s_last, states


@_on_stream
def scan_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, dy: torch.Tensor,
             states: torch.Tensor, gate: str = "sigmoid", ds_last: Optional[torch.Tensor] = None,
             grads: Optional[Sequence[torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None):
    """Gradients (dq, dk, dv, dg, ds0) of scan_fwd for upstream dy and ds_last ([B, D] fp32; None: zero).

    ``states`` is what scan_fwd returned with save_states.  dq, dk, dv, dg
    have q's type; ds0 is fp32 [B, D].  ``grads``: four tensors to write
    dq, dk, dv, dg to, sharing one row stride (slices of one [B, L, 4 D], say).
    """
    code, ld = _scan_inputs((q, k, v, g), ("q", "k", "v", "g"))
    gcode = _pick(GATES, gate, "gate")
    dev = q.device
    B, L, D = q.shape
    _contiguous(dy, "dy", (B, L, D), q.dtype, dev)
    _contiguous(states, "states", (B, -(-L // STATE_ROWS), D), torch.float32, dev)
    _contiguous(ds_last, "ds_last", (B, D), torch.float32, dev)
    if grads is None:
        grads = [torch.empty((B, L, D), dtype=q.dtype, device=dev) for _ in range(4)]
        ldd = D
    else:
        names = ("dq", "dk", "dv", "dg")
        if len(grads) != 4:
            raise ValueError("grads must be the four tensors dq, dk, dv, dg")
        ldd = _rows_like(grads, names, q.shape, q.dtype, dev)
    ds0 = torch.empty((B, D), dtype=torch.float32, device=dev)
    ws = _workspace(scan_workspace_bytes(B, L, D, code), workspace, dev)
    _call("hyena_scan_bwd", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), dy.data_ptr(),
          states.data_ptr(), _ptr(ds_last), B, L, D, ld, ldd, gcode, *(t.data_ptr() for t in grads), ds0.data_ptr(),
          *_ws_args(ws), code)
    return (*grads, ds0)


@_on_stream
def scan_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, state: torch.Tensor,
              slots: Optional[torch.Tensor] = None, gate: str = "sigmoid",
              state_out: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """y of one token for B sequences whose states are rows of ``state`` ([S, D] fp32), updated in place.

    q, k, v, g: [B, D], rows at one stride.  slots: int32 [B], the state row of
    each sequence (None: row b); one outside [0, S) marks an inactive entry
    (y = 0, no state touched).  state_out: the new states go there instead.
    """
    code = _code(q)
    gcode = _pick(GATES, gate, "gate")
    dev = q.device
    if q.dim() != 2 or state.dim() != 2:
        raise ValueError("q, k, v, g must be [B, D] and state [S, D]")
    B, D = q.shape
    ld = _rows_like((q, k, v, g), ("q", "k", "v", "g"), q.shape, q.dtype, dev)
    S = state.shape[0]
    _contiguous(state, "state", (S, D), torch.float32, dev)
    _contiguous(state_out, "state_out", (S, D), torch.float32, dev)
    _contiguous(slots, "slots", (B,), torch.int32, dev)
    if out is None:
        out = torch.empty((B, D), dtype=q.dtype, device=dev)
    else:
        _contiguous(out, "out", (B, D), q.dtype, dev)
    _call("hyena_scan_step", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), B, D, ld, gcode,
          state.data_ptr(), _ptr(state_out), S, _ptr(slots), out.data_ptr(), code)
    return out


class GatedScan(torch.autograd.Function):
    """Autograd wrapper: y, s_last = GatedScan.apply(q, k, v, g, gate, s0).  No second derivatives: they raise."""

    @staticmethod
    def forward(ctx, q, k, v, g, gate="sigmoid", s0=None):
        y, s_last, states = scan_fwd(q, k, v, g, gate=gate, s0=s0, save_states=True)
        ctx.save_for_backward(q, k, v, g, states, s0)
        ctx.gate = gate
        return y, s_last

    @staticmethod
    @first_order
    def backward(ctx, dy, ds_last):
        q, k, v, g, states, _ = ctx.saved_tensors
        need = ctx.needs_input_grad
        dq, dk, dv, dg, ds0 = scan_bwd(q, k, v, g, dy.contiguous(), states, gate=ctx.gate,
                                       ds_last=ds_last.contiguous())
        grads = (dq, dk, dv, dg, None, ds0)
        return tuple(t if n else None for t, n in zip(grads, need))  # as many as apply was given


# ---- the gated convolution, one token at a time --------------------------------------

def _cache_sizes(cache: torch.Tensor, D: int, dtype, dev):
    if cache.dim() != 3:
        raise ValueError("cache must be [S, R, D]")
    S, R = cache.shape[0], cache.shape[1]
    _contiguous(cache, "cache", (S, R, D), dtype, dev)
    return S, R


@_on_stream
def conv_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, h: torch.Tensor, cache: torch.Tensor,
              pos: torch.Tensor, group_size: int, slots: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """y = q (h * (k v)) for one token of B sequences; k v joins the ring cache.

    q, k, v: [B, D], rows at one stride; h: [D // group_size, l_h]; cache:
    [S, R, D] of the same type, R >= l_h; pos: int64 [B], the rows each
    sequence has had (the caller advances it); slots as for scan_step.
    """
    code = _code(q)
    dev = q.device
    if q.dim() != 2 or h.dim() != 2:
        raise ValueError("q, k, v must be [B, D]; h [D // group_size, l_h]")
    B, D = q.shape
    ld = _rows_like((q, k, v), ("q", "k", "v"), q.shape, q.dtype, dev)
    G, l_h = h.shape
    if group_size < 1 or D % group_size != 0 or G != D // group_size:
        raise ValueError("h has %d filters; D=%d, group_size=%d" % (G, D, group_size))
    _contiguous(h, "h", (G, l_h), q.dtype, dev)
    S, R = _cache_sizes(cache, D, q.dtype, dev)
    _contiguous(pos, "pos", (B,), torch.int64, dev)
    _contiguous(slots, "slots", (B,), torch.int32, dev)
    if out is None:
        out = torch.empty((B, D), dtype=q.dtype, device=dev)
    else:
        _contiguous(out, "out", (B, D), q.dtype, dev)
    _call("hyena_conv_step", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), h.data_ptr(), B, D, ld,
          group_size, l_h, cache.data_ptr(), S, R, pos.data_ptr(), _ptr(slots), out.data_ptr(), code)
    return out


@_on_stream
def conv_cache_fill(k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, lens: Optional[torch.Tensor] = None,
                    slots: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> None:
    """The last rows of a prompt's k v into the ring cache, for conv_step from pos = lens on.

    k, v: [B, L, D], rows at one stride; lens: int64 [B] rows of each prompt
    (None: L); cache and slots as for conv_step.
    """
    code = _code(k)
    dev = k.device
    if k.dim() != 3:
        raise ValueError("k, v must be [B, L, D]")
    B, L, D = k.shape
    ld = _rows_like((k, v), ("k", "v"), k.shape, k.dtype, dev)
    S, R = _cache_sizes(cache, D, k.dtype, dev)
    _contiguous(lens, "lens", (B,), torch.int64, dev)
    _contiguous(slots, "slots", (B,), torch.int32, dev)
    _call("hyena_conv_cache_fill", dev, k.data_ptr(), v.data_ptr(), B, L, D, ld, cache.data_ptr(), S, R,
          _ptr(lens), _ptr(slots), code)


# ---- matrix product with an epilogue --------------------------------------------------

@functools.lru_cache(maxsize=1024)
def linear_workspace_bytes(M: int, N: int, K: int, act: str = "none", dtype: int = 0, backward: bool = False) -> int:
    """Workspace bytes linear_fwd (or linear_bwd) needs."""
    n = ctypes.c_int64()
    st = layer_lib().hyena_linear_workspace(M, N, K, _pick(ACTS, act, "act"), dtype, int(backward), ctypes.byref(n))
    if st != 0:
        raise LayerError(st, "hyena_linear_workspace")
    return n.value


def _rows_of(t: torch.Tensor) -> int:
    n = 1
    for s in t.shape[:-1]:
        n *= s
    return n


@_on_stream
def linear_fwd(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
               residual: Optional[torch.Tensor] = None, act: str = "none", save_preact: bool = False,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None):
    """(y, z): z = x w^T + bias, y = act(z) + residual; z is returned with ``save_preact``, else None.

    x: [..., K], rows at one stride; w: [N, K]; bias: [N]; residual: [..., N],
    rows at one stride; all of one type.  act: none, relu, gelu (with the
    normal distribution function), silu or sigmoid.  ``out`` may be the
    residual itself.
    """
    code = _code(x)
    acode = _pick(ACTS, act, "act")
    dev, dt = x.device, x.dtype
    if x.dim() < 1 or w.dim() != 2 or x.shape[-1] != w.shape[1]:
        raise ValueError("x must be [..., K] and w [N, K]")
    N, K = w.shape
    shape = x.shape[:-1] + (N,)
    M = _rows_of(x)
    ldx = _shared_stride((x,), ("x",), K)
    _contiguous(w, "w", (N, K), dt, dev)
    _contiguous(bias, "bias", (N,), dt, dev)
    ldr = ldy = N
    if residual is not None:
        _like(residual, "residual", shape, dt, dev)
        ldr = _shared_stride((residual,), ("residual",), N)
    if out is None:
        out = torch.empty(shape, dtype=dt, device=dev)
    else:
        _like(out, "out", shape, dt, dev)
        ldy = _shared_stride((out,), ("out",), N)
    preact = torch.empty(shape, dtype=dt, device=dev) if save_preact else None
    ws = _workspace(linear_workspace_bytes(M, N, K, act, code), workspace, dev)
    _call("hyena_linear_fwd", dev, x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(residual), M, N, K, ldx, ldr,
          ldy, acode, out.data_ptr(), _ptr(preact), *_ws_args(ws), code)
    return out, preact


@_on_stream
def linear_bwd(x: torch.Tensor, w: torch.Tensor, dy: torch.Tensor, preact: Optional[torch.Tensor] = None,
               act: str = "none", need_dx: bool = True, need_dw: bool = True, need_db: bool = True,
               dx: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None):
    """Gradients (dx, dw, db) of linear_fwd for upstream dy ([..., N], rows at one stride).

    ``preact`` is the z that linear_fwd saved (not wanted for act "none").  The
    residual's gradient is dy itself.  Parts not requested are None; ``dx``
    may be given to be written to.  In bf16 with an activation dz = dy act'(z)
    is rounded to bf16 before its two products, as the matrix cores take it
    (relative errors of dx and dw 0.0024, of which 0.0017 are their own
    rounding); db sums dz as it is.
    """
    code = _code(x)
    acode = _pick(ACTS, act, "act")
    dev, dt = x.device, x.dtype
    if x.dim() < 1 or w.dim() != 2 or x.shape[-1] != w.shape[1]:
        raise ValueError("x must be [..., K] and w [N, K]")
    N, K = w.shape
    shape = x.shape[:-1] + (N,)
    M = _rows_of(x)
    ldx = _shared_stride((x,), ("x",), K)
    _contiguous(w, "w", (N, K), dt, dev)
    _like(dy, "dy", shape, dt, dev)
    lddy = _shared_stride((dy,), ("dy",), N)
    if acode != 0:
        if preact is None:
            raise ValueError("the backward of an activation needs preact")
        _contiguous(preact, "preact", shape, dt, dev)
    lddx = K
    if need_dx:
        if dx is None:
            dx = torch.empty(x.shape, dtype=dt, device=dev)
        else:
            _like(dx, "dx", x.shape, dt, dev)
            lddx = _shared_stride((dx,), ("dx",), K)
    else:
        dx = None
    dw = torch.empty((N, K), dtype=dt, device=dev) if need_dw else None
    db = torch.empty((N,), dtype=dt, device=dev) if need_db else None
    if dx is None and dw is None and db is None:
        return None, None, None
    ws = _workspace(linear_workspace_bytes(M, N, K, act, code, backward=True), workspace, dev)
    _call("hyena_linear_bwd", dev, x.data_ptr(), w.data_ptr(), _ptr(preact) if acode else None,
          dy.data_ptr(), M, N, K, ldx, lddy, lddx, acode, _ptr(dx), _ptr(dw), _ptr(db), *_ws_args(ws), code)
    return dx, dw, db


class LinearAct(torch.autograd.Function):
    """Autograd wrapper: y = LinearAct.apply(x, w, bias, residual, act); bias and residual may be None.

    No second derivatives: they raise (the residual's gradient is the incoming one and keeps its graph).
    """

    @staticmethod
    def forward(ctx, x, w, bias=None, residual=None, act="none"):
        y, z = linear_fwd(x, w, bias=bias, residual=residual, act=act, save_preact=act != "none")
        ctx.save_for_backward(x, w, z, bias)
        ctx.act = act
        return y

    @staticmethod
    @first_order
    def backward(ctx, dy):
        x, w, z, _ = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = linear_bwd(x, w, dy.contiguous(), preact=z, act=ctx.act, need_dx=need[0], need_dw=need[1],
                                need_db=len(need) > 2 and need[2])
        grads = (dx, dw, db, dy, None)
        return tuple(t if n else None for t, n in zip(grads, need))  # as many as apply was given
