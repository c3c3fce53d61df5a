"""C-ABI contract of include/hyena_model.h, without a GPU: exports, and refusals before any HIP call.

The addresses are fake and never dereferenced: a rejected call touches no device."""
import ctypes
import math
import os
import re

import pytest

import gated_convolution_sequence_amd as hc
from gated_convolution_sequence_amd.model import _Tensor

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
G = 1 << 40
P = [G + (i << 36) for i in range(20)]  # far apart
WS = 1 << 34  # a workspace no size here outgrows


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(hc.MODEL_LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return hc.model_lib()


def test_header_declares_the_python_export_list():
    text = open(os.path.join(ROOT, "include", "hyena_model.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    assert sorted(set(re.findall(r"\b(hyena_\w+)\s*\(", text))) == sorted(hc.MODEL_EXPORTS)
    lib = ctypes.CDLL(hc.MODEL_LIB_PATH)
    for name in hc.MODEL_EXPORTS:
        assert hasattr(lib, name), name


def test_every_status_has_a_text():
    for code in list(hc.STATUS) + [-100, 7]:
        assert hc.model_strerror(code)
    assert hc.model_strerror(0) == "ok"
    err = hc.ModelError(-2, "here")
    assert isinstance(err, hc.HyenaError) and err.status == -2 and "here" in str(err)


def norm_fwd(x=P[0], w=P[1], b=P[2], M=5, D=64, ldx=64, ldy=64, kind=0, eps=1e-5, y=P[3], mean=P[4], rstd=P[5], dtype=0):
    return hc.model_lib().hyena_norm_fwd(x, w, b, M, D, ldx, ldy, kind, eps, y, mean, rstd, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(y=None), -1),
    (dict(M=-1), -2), (dict(D=-1), -2), (dict(ldx=63), -2), (dict(ldy=63), -2), (dict(ldx=1 << 62), -2),
    (dict(M=1 << 40, D=1 << 30, ldx=1 << 30, ldy=1 << 30), -2), (dict(D=1 << 32, ldx=1 << 32, ldy=1 << 32), -2),
    (dict(x=P[0] + 1), -5), (dict(dtype=1, w=P[1] + 2), -5), (dict(b=P[2] + 1), -5), (dict(mean=P[4] + 2), -5),
    (dict(rstd=P[5] + 1), -5),
    (dict(y=P[0]), -6), (dict(y=P[1]), -6), (dict(mean=P[5]), -6), (dict(rstd=P[3] + 64), -6), (dict(ldx=128, y=P[0] + 64), -6),
    (dict(kind=2), -7), (dict(kind=-1), -7), (dict(kind=1), -7), (dict(eps=-1.0), -7), (dict(eps=math.nan), -7),
    (dict(eps=math.inf), -7), (dict(dtype=2), -9),
])
def test_norm_fwd_refusals(kw, code):
    assert norm_fwd(**kw) == code


def norm_bwd(x=P[0], w=P[1], dy=P[2], mean=P[3], rstd=P[4], M=5, D=64, ldx=64, lddy=64, lddx=64, kind=0, dx=P[5],
             dw=P[6], db=P[7], ws=P[8], n=WS, dtype=0):
    return hc.model_lib().hyena_norm_bwd(x, w, dy, mean, rstd, M, D, ldx, lddy, lddx, kind, dx, dw, db, ws, n, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(dy=None), -1), (dict(mean=None), -1), (dict(rstd=None), -1),
    (dict(dx=None, dw=None, db=None), -1),
    (dict(M=-1), -2), (dict(D=-3), -2), (dict(lddy=63), -2), (dict(lddx=63), -2), (dict(lddx=1 << 62), -2),
    (dict(dy=P[2] + 1), -5), (dict(dx=P[5] + 1), -5), (dict(ws=P[8] + 8), -5), (dict(mean=P[3] + 2), -5),
    (dict(dx=P[0]), -6), (dict(dx=P[2]), -6), (dict(dw=P[1]), -6), (dict(db=P[6] + 64), -6), (dict(ws=P[4]), -6),
    (dict(kind=1), -7), (dict(kind=3), -7), (dict(dtype=5), -9), (dict(ws=None, n=0), -10), (dict(n=16), -10),
])
def test_norm_bwd_refusals(kw, code):
    assert norm_bwd(**kw) == code


def xent_fwd(x=P[0], w=P[1], bias=P[2], target=P[3], M=40, K=64, V=100, ldx=64, loss=P[4], lse=P[5], ws=P[6], n=WS, dtype=0):
    return hc.model_lib().hyena_xent_fwd(x, w, bias, target, M, K, V, ldx, loss, lse, ws, n, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(w=None), -1), (dict(target=None), -1), (dict(loss=None), -1), (dict(lse=None), -1),
    (dict(M=-1), -2), (dict(K=-1), -2), (dict(V=-1), -2), (dict(V=0), -2), (dict(ldx=63), -2), (dict(V=1 << 31), -2),
    (dict(M=1 << 31), -2), (dict(ldx=1 << 62), -2), (dict(K=1 << 20, ldx=1 << 20), -7),
    (dict(x=P[0] + 1), -5), (dict(target=P[3] + 4), -5), (dict(loss=P[4] + 2), -5), (dict(ws=P[6] + 8), -5),
    (dict(dtype=1, bias=P[2] + 2), -5),
    (dict(loss=P[5]), -6), (dict(lse=P[3]), -6), (dict(loss=P[0]), -6), (dict(ws=P[1]), -6), (dict(ws=P[4]), -6),
    (dict(dtype=2), -9), (dict(ws=None, n=0), -10), (dict(n=64), -10),
])
def test_xent_fwd_refusals(kw, code):
    assert xent_fwd(**kw) == code


def xent_bwd(x=P[0], w=P[1], bias=P[2], target=P[3], lse=P[4], dloss=P[5], M=40, K=64, V=100, ldx=64, lddx=64, dx=P[6],
             dw=P[7], db=P[8], ws=P[9], n=WS, dtype=0):
    return hc.model_lib().hyena_xent_bwd(x, w, bias, target, lse, dloss, M, K, V, ldx, lddx, dx, dw, db, ws, n, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(w=None), -1), (dict(target=None), -1), (dict(lse=None), -1), (dict(dloss=None), -1),
    (dict(dx=None, dw=None, db=None), -1),
    (dict(M=-1), -2), (dict(V=0), -2), (dict(ldx=63), -2), (dict(lddx=63), -2), (dict(lddx=1 << 62), -2),
    (dict(lse=P[4] + 2), -5), (dict(dloss=P[5] + 2), -5), (dict(dx=P[6] + 1), -5), (dict(dw=P[7] + 1), -5),
    (dict(dx=P[0]), -6), (dict(dw=P[1]), -6), (dict(db=P[2]), -6), (dict(dx=P[5]), -6), (dict(db=P[7]), -6),
    (dict(ws=P[6]), -6), (dict(dtype=3), -9), (dict(n=1000), -10),
])
def test_xent_bwd_refusals(kw, code):
    assert xent_bwd(**kw) == code


def test_workspaces_are_checked_where_one_is_needed():
    for call, kw, n in ((norm_bwd, {}, hc.norm_workspace_bytes(5, 64)),
                        (xent_fwd, {}, hc.xent_workspace_bytes(40, 64, 100)),
                        (xent_fwd, dict(M=3), hc.xent_workspace_bytes(3, 64, 100)),
                        (xent_bwd, {}, hc.xent_workspace_bytes(40, 64, 100, backward=True))):
        assert n > 0 and call(n=n - 1, **kw) == -10 and call(n=n, ws=P[0], **kw) == -6
    lib = hc.model_lib()
    assert lib.hyena_norm_workspace(1, 1, 0, None) == -1 and lib.hyena_xent_workspace(1, 1, 1, 0, 0, None) == -1
    assert lib.hyena_grad_norm_workspace(1, 1, None) == -1
    assert lib.hyena_norm_workspace(-1, 1, 0, None) == -2 and lib.hyena_grad_norm_workspace(-1, 1, None) == -2
    with pytest.raises(hc.ModelError):
        hc.xent_workspace_bytes(1, 1 << 21, 1)


def test_no_logits_in_the_workspace():
    """The forward's workspace grows with the rows and the tiles, the backward's by a piece of the vocabulary."""
    M, K, V = 8192, 4096, 1 << 18
    assert hc.xent_workspace_bytes(M, K, V) < M * V // 4
    assert hc.xent_workspace_bytes(M, K, V, backward=True) < M * V * 2 // 4


def tensors(*rows):
    table = (_Tensor * max(1, len(rows)))()
    for e, r in zip(table, rows):
        for k, v in r.items():
            setattr(e, k, v)
    return table


ROW = dict(param=P[0], grad=P[1], exp_avg=P[2], exp_avg_sq=P[3], exp_avg_scale=P[4], exp_avg_sq_scale=P[5], master=P[6],
           numel=1000)


def adamw(rows=(ROW,), n=None, lr=1e-3, b1=0.9, b2=0.95, eps=1e-8, decay=0.1, step=1, seed=0, lr_dev=None, step_dev=None,
          seed_dev=None, scale=P[7], bits=32, dtype=0, table=True):
    t = tensors(*rows)
    return hc.model_lib().hyena_adamw_step(ctypes.addressof(t) if table else None, len(rows) if n is None else n, lr, b1,
                                           b2, eps, decay, step, seed, lr_dev, step_dev, seed_dev, scale, bits, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(table=False), -1), (dict(n=-1), -2), (dict(rows=({**ROW, "numel": -1},)), -2),
    (dict(rows=({**ROW, "numel": 1 << 40},)), -2),
    *((dict(rows=({**ROW, name: None},)), -1) for name in ("param", "grad", "exp_avg", "exp_avg_sq")),
    *((dict(rows=({**ROW, name: None},), bits=8), -1) for name in ("exp_avg_scale", "exp_avg_sq_scale")),
    (dict(rows=({**ROW, "param": P[0] + 1},)), -5), (dict(rows=({**ROW, "exp_avg": P[2] + 2},)), -5),
    (dict(rows=({**ROW, "master": P[6] + 2},)), -5), (dict(rows=({**ROW, "exp_avg_scale": P[4] + 2},), bits=8), -5),
    (dict(rows=(ROW, {**ROW, "grad": P[1] + 1})), -5), (dict(scale=P[7] + 2), -5), (dict(lr_dev=P[8] + 2), -5),
    (dict(step_dev=P[8] + 4), -5), (dict(seed_dev=P[8] + 4), -5),
    (dict(rows=({**ROW, "master": P[2]},)), -6), (dict(rows=({**ROW, "grad": P[0]},)), -6),
    (dict(rows=({**ROW, "exp_avg_scale": P[5]},), bits=8), -6), (dict(rows=({**ROW, "exp_avg_sq": P[2] + 3996},)), -6),
    (dict(rows=(ROW, ROW)), -6),
    (dict(rows=(ROW, {**{k: v + 4096 for k, v in ROW.items()}, "numel": 1000, "exp_avg": P[3] + 3996})), -6),
    (dict(rows=(ROW, {**{k: v + 4096 for k, v in ROW.items()}, "numel": 1000, "grad": P[6]})), -6),
    (dict(scale=P[2] + 40), -6), (dict(step_dev=P[6]), -6),
    (dict(lr=math.nan), -7), (dict(b1=1.0), -7), (dict(b1=-0.1), -7), (dict(b2=1.0), -7), (dict(b2=math.nan), -7),
    (dict(eps=-1e-8), -7), (dict(eps=math.inf), -7), (dict(decay=math.inf), -7), (dict(step=0), -7), (dict(bits=16), -7),
    (dict(dtype=2), -9),
])
def test_adamw_refusals(kw, code):
    assert adamw(**kw) == code


def grad_norm(rows=(ROW,), n=None, max_norm=1.0, norm=P[8], scale=P[9], ws=P[10], size=WS, dtype=0, table=True):
    t = tensors(*rows)
    return hc.model_lib().hyena_grad_norm(ctypes.addressof(t) if table else None, len(rows) if n is None else n, max_norm,
                                          norm, scale, ws, size, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(table=False), -1), (dict(norm=None), -1), (dict(rows=({**ROW, "grad": None},)), -1), (dict(n=-1), -2),
    (dict(norm=P[8] + 2), -5), (dict(scale=P[9] + 2), -5), (dict(ws=P[10] + 8), -5), (dict(rows=({**ROW, "grad": P[1] + 1},)), -5),
    (dict(scale=P[8]), -6), (dict(norm=P[1] + 400), -6), (dict(ws=P[1]), -6), (dict(ws=P[8]), -6),
    (dict(max_norm=-1.0), -7), (dict(max_norm=math.nan), -7), (dict(dtype=2), -9), (dict(size=0), -10), (dict(ws=None), -10),
])
def test_grad_norm_refusals(kw, code):
    assert grad_norm(**kw) == code


def test_nothing_to_do_needs_no_pointers():
    assert norm_fwd(M=0, x=None, y=None, w=None, b=None, mean=None, rstd=None) == 0
    assert norm_fwd(D=0, ldx=0, ldy=0, x=None, y=None, w=None, b=None, mean=None, rstd=None) == 0
    assert norm_bwd(D=0, ldx=0, lddy=0, lddx=0, x=None, dy=None, dx=None, dw=None, db=None, ws=None, n=0) == 0
    assert norm_bwd(M=0, x=None, dy=None, mean=None, rstd=None, dx=None, dw=None, db=None, ws=None, n=0) == 0
    assert xent_fwd(M=0, x=None, target=None, loss=None, lse=None, ws=None, n=0) == 0
    assert xent_bwd(M=0, x=None, target=None, lse=None, dloss=None, dx=None, dw=None, db=None, ws=None, n=0) == 0
    assert adamw(rows=()) == 0 and adamw(rows=({**ROW, "numel": 0, "grad": None},)) == 0
