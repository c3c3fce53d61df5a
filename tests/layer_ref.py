"""Plain 64-bit implementations of the sequence-layer operators, with error bounds (CPU, numpy).

Bounds follow the operators' stated precision: fp32 gates, states and sums,
one rounding of each output to its type.  u = 2^-23 bounds a correctly or
nearly correctly rounded fp32 operation (at most one unit in the last place).

Recurrence.  A decay is off by at most (|g| + 6) u relative (|g| u for the
rounding of the exponent's argument, the rest for exp, the reciprocal and the
products).  Walking or joining partial sums in any order multiplies each
term's factor by at most one extra rounded product and one rounded sum a row,
so with the recurrence sbar on magnitudes the error obeys
    E_t <= a_t (E_{t-1} + (|g_t| + 10) u sbar_{t-1}) + 4 u sbar_t.
"""
import math

import numpy as np
import torch

U = 2.0 ** -23
TINY = 1e-36


def to_np(t):
    return t.detach().to("cpu", torch.float64).numpy()


def out_rounding(dtype):
    """Relative rounding of an output: one unit in the last place of its type."""
    return 2.0 ** -8 if dtype == torch.bfloat16 else U


def check(got, ref, bound, dtype, what):
    """|got - ref| <= bound + the output's rounding; non-finite values in the same places."""
    got = to_np(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    fin = np.isfinite(ref)
    assert np.array_equal(fin, np.isfinite(got)), "%s: non-finite values differ" % what
    assert np.array_equal(np.isnan(ref), np.isnan(got)), "%s: NaN differ" % what
    assert np.array_equal(ref[~fin & ~np.isnan(ref)], got[~fin & ~np.isnan(ref)]), "%s: infinities differ" % what
    with np.errstate(invalid="ignore", over="ignore"):
        bad = fin & (np.abs(got - ref) > bound + out_rounding(dtype) * np.abs(ref) + TINY)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError("%s: %d of %d off, first at %s: got %r, ref %r, bound %r" % (
            what, bad.sum(), bad.size, i, got[i], ref[i], np.broadcast_to(bound, ref.shape)[i]))


def decay(g, gate):
    """(a, da/dg) in 64 bits."""
    with np.errstate(over="ignore"):
        if gate == "log":
            a = np.exp(g)
            return a, a
        e = np.exp(-np.abs(g))
        return np.where(g < 0, e / (1 + e), 1 / (1 + e)), e / (1 + e) ** 2


def _walk(a, x, first):
    """All s_t = a_t s_{t-1} + x_t along axis 1; where a_t is 0 the state before is dropped."""
    s, out = first, np.empty_like(x)
    for t in range(x.shape[1]):
        with np.errstate(invalid="ignore", over="ignore"):
            s = np.where(a[:, t] == 0, 0.0, a[:, t] * s) + x[:, t]
        out[:, t] = s
    return out


def _walk_error(a, ga, sbar, sbar0):
    """E of the module's note."""
    prev = np.concatenate([sbar0[:, None], sbar[:, :-1]], axis=1)
    with np.errstate(invalid="ignore", over="ignore"):
        x = np.where(a == 0, 0.0, a * (ga + 10) * U * prev) + 4 * U * sbar
    return _walk(a, x, np.zeros_like(sbar0))


def scan_fwd(q, k, v, g, gate, s0=None):
    """y, s, states (64 rows apart) and bounds for y and s; numpy [B, L, D], s0 [B, D] or None."""
    B, L, D = q.shape
    s0 = np.zeros((B, D)) if s0 is None else s0
    a, _ = decay(g, gate)
    ga = np.where(np.isfinite(g), np.abs(g), 0.0)
    x = k * v
    s = _walk(a, x, s0)
    sbar = _walk(a, np.abs(x), np.abs(s0))
    es = _walk_error(a, ga, sbar, np.abs(s0))
    full = np.concatenate([s0[:, None], s], axis=1)
    efull = np.concatenate([np.zeros((B, 1, D)), es], axis=1)
    return dict(y=q * s, ey=np.abs(q) * es + U * np.abs(q) * sbar, s=s, es=es, last=full[:, -1], elast=efull[:, -1],
                states=full[:, 0:L:64], estates=efull[:, 0:L:64], prev=full[:, :-1], eprev=efull[:, :-1],
                a=a, ga=ga, sbar=sbar)


def scan_bwd(q, k, v, g, dy, gate, s0=None, ds_last=None):
    """Gradients and their bounds: dict name -> (ref, bound) for dq, dk, dv, dg, ds0."""
    B, L, D = q.shape
    f = scan_fwd(q, k, v, g, gate, s0)
    a, ga = f["a"], f["ga"]
    _, slope = decay(g, gate)
    first = np.zeros((B, D)) if ds_last is None else ds_last
    u = q * dy
    nxt = np.concatenate([a[:, 1:], np.ones((B, min(L, 1), D))], axis=1)[:, ::-1]
    gn = np.concatenate([ga[:, 1:], np.zeros((B, min(L, 1), D))], axis=1)[:, ::-1]
    ds = _walk(nxt, u[:, ::-1], first)[:, ::-1]
    dbar = _walk(nxt, np.abs(u)[:, ::-1], np.abs(first))
    ed = _walk_error(nxt, gn, dbar, np.abs(first))[:, ::-1]
    dbar = dbar[:, ::-1]
    with np.errstate(invalid="ignore", over="ignore"):
        dg = np.where(a == 0, 0.0, ds * f["prev"] * slope)
        edg = np.where(a == 0, 0.0, slope * (np.abs(ds) * f["eprev"] + np.abs(f["prev"]) * ed
                                             + (2 * ga + 12) * U * dbar * np.abs(f["prev"])))
        c0 = np.where(a[:, 0] == 0, 0.0, a[:, 0] * ds[:, 0]) if L else first
        e0 = np.where(a[:, 0] == 0, 0.0, a[:, 0] * (ed[:, 0] + (ga[:, 0] + 8) * U * dbar[:, 0])) if L else 0 * first
    return dict(dq=(dy * f["s"], np.abs(dy) * (f["es"] + U * f["sbar"])),
                dk=(ds * v, np.abs(v) * (ed + U * dbar)), dv=(ds * k, np.abs(k) * (ed + U * dbar)),
                dg=(dg, edg), ds0=(c0, e0))


# ---- linear -----------------------------------------------------------------------

# largest slope of each activation
LIPSCHITZ = {"none": 1.0, "relu": 1.0, "gelu": 1.13, "silu": 1.1, "sigmoid": 0.25}


def act(z, name):
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "gelu":
        return 0.5 * z * (1 + _erf(z / math.sqrt(2)))
    with np.errstate(over="ignore"):
        if name == "silu":
            return z / (1 + np.exp(-z))
        if name == "sigmoid":
            return 1 / (1 + np.exp(-z))
    return z


def _erf(x):
    return torch.erf(torch.from_numpy(np.ascontiguousarray(x))).numpy()


def act_slope(z, name):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return 0.5 * (1 + _erf(z / math.sqrt(2))) + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name in ("silu", "sigmoid"):
        p, s = decay(z, "sigmoid")
        return p + z * s if name == "silu" else s
    return np.ones_like(z)


def linear_fwd(x, w, bias, residual, name):
    """y, z and bounds.  A sum of n products in any order is off by at most (n + 8) u of its terms' magnitudes."""
    K = x.shape[1]
    z = x @ w.T
    ez = (K + 8) * U * (np.abs(x) @ np.abs(w).T)
    if bias is not None:
        z = z + bias
        ez = ez + U * np.abs(bias)
    y = act(z, name)
    ey = LIPSCHITZ[name] * ez + (0 if name == "none" else 16 * U * (1 + np.abs(z)))
    if residual is not None:
        ey = ey + U * (np.abs(y) + np.abs(residual))
        y = y + residual
    return y, ey, z, ez


def linear_bwd(x, w, z, dy, name, bf16):
    """dx, dw, db with bounds.  bf16: dz is rounded once as an operand (one unit, 2^-8), but not for db."""
    M, N = dy.shape
    slope = act_slope(z, name) if name != "none" else np.ones_like(dy)
    dz = dy * slope
    e = 0.0 if name == "none" else np.abs(dy) * 32 * U * (1 + z * z)
    # a sum's own rounding, and the rounding of the operand
    op = np.abs(dz) * (2.0 ** -8 if bf16 and name != "none" else 0.0) + e
    dx, dw, db = dz @ w, dz.T @ x, dz.sum(0)
    edx = (N + 8) * U * (np.abs(dz) @ np.abs(w)) + op @ np.abs(w)
    edw = (M + 8) * U * (np.abs(dz).T @ np.abs(x)) + op.T @ np.abs(x)
    edb = (M + 8) * U * np.abs(dz).sum(0) + (e if name != "none" else 0 * dz).sum(0)
    return (dx, edx), (dw, edw), (db, edb)
