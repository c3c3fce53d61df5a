"""C-ABI contract of include/hyena_layer.h, without a GPU: exports, and refusals before any HIP call.

The addresses are fake and never dereferenced: a rejected call touches no device."""
import ctypes
import os
import re

import pytest

import gated_convolution_sequence_amd as hc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
G = 1 << 40
P = [G + (i << 36) for i in range(20)]  # far apart


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(hc.LAYER_LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return hc.layer_lib()


def test_header_declares_the_python_export_list():
    text = open(os.path.join(ROOT, "include", "hyena_layer.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    assert sorted(set(re.findall(r"\b(hyena_\w+)\s*\(", text))) == sorted(hc.LAYER_EXPORTS)
    lib = ctypes.CDLL(hc.LAYER_LIB_PATH)
    for name in hc.LAYER_EXPORTS:
        assert hasattr(lib, name), name


def test_every_status_has_a_text():
    for code in list(hc.STATUS) + [-100, 7]:
        assert hc.layer_strerror(code)
    assert hc.layer_strerror(0) == "ok"


WS = 1 << 34  # a workspace no size here outgrows


def scan_fwd(q=P[0], k=P[1], v=P[2], g=P[3], B=2, L=100, D=64, ld=64, gate=0, s0=P[4], y=P[5], last=P[6],
             states=P[7], ws=P[8], n=WS, dtype=0):
    return hc.layer_lib().hyena_scan_fwd(q, k, v, g, B, L, D, ld, gate, s0, y, last, states, ws, n, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(g=None), -1),
    (dict(y=None, last=None, states=None), -1),
    (dict(B=-1), -2), (dict(L=-1), -2), (dict(D=-1), -2), (dict(ld=63), -2), (dict(L=1 << 39, D=1 << 29, ld=1 << 29), -2),
    (dict(ld=1 << 62), -2),
    (dict(q=P[0] + 1), -5), (dict(s0=P[4] + 2), -5), (dict(y=P[5] + 1), -5), (dict(ws=P[8] + 8), -5),
    (dict(dtype=1, g=P[3] + 2), -5), (dict(states=P[7] + 1), -5),
    (dict(y=P[0]), -6), (dict(y=P[3] + 128), -6), (dict(last=P[4]), -6), (dict(states=P[1]), -6),
    (dict(last=P[5]), -6), (dict(ld=128, y=P[0] + 64), -6),
    (dict(gate=2), -7), (dict(gate=-1), -7), (dict(dtype=2), -9),
])
def test_scan_fwd_refusals(kw, code):
    assert scan_fwd(**kw) == code


def scan_bwd(q=P[0], k=P[1], v=P[2], g=P[3], dy=P[4], states=P[5], last=P[6], B=2, L=100, D=64, ld=64, ldd=64, gate=0,
             dq=P[7], dk=P[8], dv=P[9], dg=P[10], ds0=P[11], ws=P[12], n=WS, dtype=0):
    return hc.layer_lib().hyena_scan_bwd(q, k, v, g, dy, states, last, B, L, D, ld, ldd, gate, dq, dk, dv, dg, ds0,
                                         ws, n, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(dy=None), -1), (dict(states=None), -1),
    (dict(dq=None, dk=None, dv=None, dg=None, ds0=None), -1),
    (dict(ldd=63), -2), (dict(B=-2), -2), (dict(ldd=1 << 62), -2),
    (dict(dq=P[7] + 1), -5), (dict(states=P[5] + 2), -5), (dict(ds0=P[11] + 2), -5),
    (dict(dq=P[0]), -6), (dict(dg=P[4] + 64), -6), (dict(dk=P[7] + 128), -6), (dict(ds0=P[6]), -6),
    # slices of one buffer that share a column
    (dict(ldd=256, dk=P[7] + 126), -6),
    (dict(gate=5), -7), (dict(dtype=-1), -9),
])
def test_scan_bwd_refusals(kw, code):
    assert scan_bwd(**kw) == code


def test_workspaces_are_checked_where_one_is_needed():
    n = hc.scan_workspace_bytes(2, 5000, 64)
    assert n >= 0 and hc.scan_workspace_bytes(0, 5, 64) == 0
    if n:
        assert scan_fwd(L=5000, n=n - 1) == -10 and scan_fwd(L=5000, ws=None, n=0) == -10
        assert scan_bwd(L=5000, n=n - 1) == -10
        assert scan_fwd(L=5000, ws=P[0], n=n) == -6
    lib = hc.layer_lib()
    assert lib.hyena_scan_workspace(1, 1, 1, 0, None) == -1
    assert lib.hyena_linear_workspace(1, 1, 1, 0, 0, 0, None) == -1
    for act in hc.ACTS:
        n = hc.linear_workspace_bytes(1000, 256, 256, act, 0, backward=True)
        if n:
            assert linear_bwd(M=1000, N=256, K=256, ldx=256, lddy=256, lddx=256, act=hc.ACTS[act], n=n - 1) == -10


def scan_step(q=P[0], k=P[1], v=P[2], g=P[3], B=2, D=64, ld=64, gate=0, state=P[4], out=P[5], S=4, slots=P[6], y=P[7],
              dtype=0):
    return hc.layer_lib().hyena_scan_step(q, k, v, g, B, D, ld, gate, state, out, S, slots, y, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(state=None), -1), (dict(y=None), -1),
    (dict(B=-1), -2), (dict(ld=63), -2), (dict(S=-1), -2), (dict(S=1, slots=None), -2),
    (dict(S=1 << 40, D=1 << 30, ld=1 << 30), -2),
    (dict(state=P[4] + 2), -5), (dict(slots=P[6] + 2), -5),
    (dict(y=P[0]), -6), (dict(y=P[4]), -6), (dict(out=P[4] + 256), -6), (dict(out=P[6]), -6),
    (dict(gate=9), -7), (dict(dtype=3), -9),
])
def test_scan_step_refusals(kw, code):
    assert scan_step(**kw) == code


def conv_step(q=P[0], k=P[1], v=P[2], h=P[3], B=2, D=64, ld=64, gs=16, l_h=7, cache=P[4], S=4, R=8, pos=P[5],
              slots=P[6], y=P[7], dtype=0):
    return hc.layer_lib().hyena_conv_step(q, k, v, h, B, D, ld, gs, l_h, cache, S, R, pos, slots, y, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(h=None), -1), (dict(cache=None), -1), (dict(pos=None), -1),
    (dict(ld=1), -2), (dict(R=6), -2), (dict(slots=None, S=1), -2), (dict(S=1 << 50, R=1 << 20), -2),
    (dict(gs=0), -3), (dict(gs=48), -3), (dict(l_h=0), -4), (dict(l_h=129, R=200), -4),
    (dict(R=1 << 25), -7), (dict(S=1 << 31), -7), (dict(S=0, R=1 << 60), -2),
    (dict(pos=P[5] + 4), -5), (dict(cache=P[4] + 1), -5),
    (dict(y=P[4]), -6), (dict(cache=P[3]), -6), (dict(y=P[5]), -6), (dict(dtype=7), -9),
])
def test_conv_step_refusals(kw, code):
    assert conv_step(**kw) == code


def cache_fill(k=P[0], v=P[1], B=2, L=10, D=64, ld=64, cache=P[2], S=4, R=8, lens=P[3], slots=P[4], dtype=0):
    return hc.layer_lib().hyena_conv_cache_fill(k, v, B, L, D, ld, cache, S, R, lens, slots, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), -1), (dict(cache=None), -1), (dict(R=0), -2), (dict(ld=2), -2), (dict(L=-1), -2),
    (dict(lens=P[3] + 4), -5), (dict(cache=P[1]), -6), (dict(dtype=2), -9),
])
def test_cache_fill_refusals(kw, code):
    assert cache_fill(**kw) == code


def linear_fwd(x=P[0], w=P[1], b=P[2], r=P[3], M=100, N=64, K=32, ldx=32, ldr=64, ldy=64, act=0, y=P[4], z=P[5],
               ws=P[6], n=WS, dtype=0):
    return hc.layer_lib().hyena_linear_fwd(x, w, b, r, M, N, K, ldx, ldr, ldy, act, y, z, ws, n, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(w=None), -1), (dict(y=None), -1),
    (dict(M=-1), -2), (dict(ldx=31), -2), (dict(ldr=63), -2), (dict(ldy=63), -2), (dict(M=1 << 31), -2),
    (dict(x=P[0] + 1), -5), (dict(dtype=1, b=P[2] + 2), -5),
    (dict(y=P[0]), -6), (dict(z=P[1]), -6), (dict(z=P[4]), -6), (dict(y=P[3] + 128), -6), (dict(y=P[3], ldy=70), -6),
    (dict(act=5), -7), (dict(act=-1), -7), (dict(dtype=2), -9),
])
def test_linear_fwd_refusals(kw, code):
    assert linear_fwd(**kw) == code


def linear_bwd(x=P[0], w=P[1], z=P[2], dy=P[3], M=100, N=64, K=32, ldx=32, lddy=64, lddx=32, act=3, dx=P[4], dw=P[5],
               db=P[6], ws=P[7], n=WS, dtype=0):
    return hc.layer_lib().hyena_linear_bwd(x, w, z, dy, M, N, K, ldx, lddy, lddx, act, dx, dw, db, ws, n, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(w=None), -1), (dict(z=None), -1), (dict(dy=None), -1),
    (dict(dx=None, dw=None, db=None), -1),
    (dict(lddy=63), -2), (dict(lddx=31), -2), (dict(N=-1), -2),
    (dict(db=P[6] + 1), -5), (dict(dx=P[0]), -6), (dict(dw=P[1]), -6), (dict(db=P[2]), -6), (dict(dw=P[4]), -6),
    (dict(act=6), -7), (dict(dtype=2), -9),
])
def test_linear_bwd_refusals(kw, code):
    assert linear_bwd(**kw) == code


def test_empty_problems_are_accepted():
    assert scan_fwd(B=0) == 0 and scan_fwd(D=0) == 0 and scan_bwd(B=0) == 0 and scan_step(B=0) == 0
    assert conv_step(B=0) == 0 and cache_fill(L=0) == 0 and linear_fwd(M=0) == 0 and linear_fwd(N=0) == 0


def test_binding_raises_with_status():
    with pytest.raises(hc.LayerError) as e:
        hc.scan_workspace_bytes(-1, 2, 3)
    assert e.value.status == -2
    with pytest.raises(hc.LayerError):
        hc.linear_workspace_bytes(1, 2, -3)
    with pytest.raises(ValueError):
        hc.linear_workspace_bytes(1, 2, 3, act="tanh")
