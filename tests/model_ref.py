"""Plain 64-bit implementations of the model operators, with error bounds (torch, on the inputs' device).

As tests/layer_ref.py: U = 2^-23 bounds an fp32 operation's relative error, and
check() adds the output's one rounding.  A sum of n terms made of lanes, steps
between lanes and workgroups rounds each term at most depth(n) times.  The hardware's exp(x)
is off by (|x| + 2) U: the argument's product with log2 e is rounded, and so is the result.
"""
import torch

from layer_ref import U

F64 = torch.float64


def check(got, ref, bound, what):
    """|got - ref| <= bound + half a unit of got's type; non-finite values in the same places."""
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    x = got.double()
    fine = torch.isfinite(ref)
    assert torch.equal(fine, torch.isfinite(x)), what + ": other values are finite"
    same = (x == ref) | (torch.isnan(x) & torch.isnan(ref))
    assert bool((same | fine).all()), what + ": other infinities or NaN"
    half = torch.finfo(got.dtype).eps / 2
    err = torch.where(fine, (x - ref).abs() - ref.abs() * half, 0.0)
    slack = torch.where(fine, bound, 0.0) + 1e-37  # below fp32's and bf16's normal range
    worst = (err - slack).max() if err.numel() else torch.tensor(0.0)
    assert float(worst) <= 0, "%s: off by %.3e beyond %.3e" % (what, float(err.max()), float(slack.max()))


def depth(n):
    """Roundings that a term of a norm's row sum of n sees: 64 values a lane or a loop's turns, then lanes and waves."""
    return 96 + n / 1024


# ---- norm ---------------------------------------------------------------------------

def norm_fwd(x, w, b, kind, eps):
    """y, mean, rstd as (ref, bound) each; x [M, D]."""
    x = x.double()
    D = x.shape[1]
    n = depth(D)
    w = torch.ones(D, dtype=F64, device=x.device) if w is None else w.double()
    b = torch.zeros(D, dtype=F64, device=x.device) if b is None else b.double()
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    em = n * U * x.abs().mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(mean)
    d = x - mean
    var = (d * d).mean(1, keepdim=True)
    ed = em + U * d.abs()
    evar = (n + 4) * U * var + 2 * (ed * d.abs()).mean(1, keepdim=True) + (ed * ed).mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    # the least that var + eps can have come to: its reciprocal root's error to all orders
    low = (var + eps - evar - U * (var + eps)).clamp(min=1e-300)
    er = (low ** -0.5 - rstd) + 4 * U * rstd
    y = d * rstd * w + b
    ey = w.abs() * (rstd * ed + d.abs() * er + ed * er) + 4 * U * (d * rstd * w).abs() + U * y.abs()
    return (y, ey), (mean[:, 0], em[:, 0] + U * mean[:, 0].abs()), (rstd[:, 0], er[:, 0])


def norm_bwd(x, w, dy, mean, rstd, kind):
    """dx, dw, db as (ref, bound) from the saved statistics."""
    x, dy, r = x.double(), dy.double(), rstd.double()[:, None]
    M, D = x.shape
    n = depth(D)
    w = torch.ones(D, dtype=F64, device=x.device) if w is None else w.double()
    u = x * r if kind == "rms" else (x - mean.double()[:, None]) * r
    eu = 3 * U * u.abs()
    g = w * dy
    c1 = (g * u).mean(1, keepdim=True)
    ec1 = (n + 6) * U * (g * u).abs().mean(1, keepdim=True)
    c0 = g.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(c1)
    ec0 = (n + 2) * U * g.abs().mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(c1)
    dx = r * (g - c0 - u * c1)
    edx = r.abs() * (4 * U * (g.abs() + c0.abs() + (u * c1).abs()) + ec0 + u.abs() * ec1 + eu * c1.abs()) + 2 * U * dx.abs()
    rows = min(M, 160 + M / 128)  # a lane's rows, then the workgroups'
    dw, db = (dy * u).sum(0), dy.sum(0)
    return (dx, edx), (dw, (rows + 6) * U * (dy * u).abs().sum(0)), (db, (rows + 2) * U * dy.abs().sum(0))


# ---- softmax cross entropy --------------------------------------------------------------

def logits(x, w, bias):
    x, w = x.double(), w.double()
    z = x @ w.t()
    ez = (x.shape[1] + 8) * U * (x.abs() @ w.abs().t())
    if bias is not None:
        z = z + bias.double()
        ez = torch.where(torch.isfinite(z), ez + U * z.abs(), 0.0)
    return z, ez


def xent_fwd(x, w, target, bias):
    """loss, lse as (ref, bound); rows without a target are taken out before anything is computed."""
    V = w.shape[0]
    on = (target >= 0) & (target < V)
    rows = torch.nonzero(on)[:, 0]
    out = [torch.zeros(target.shape, dtype=F64, device=x.device) for _ in range(4)]
    if len(rows):
        z, ez = logits(x[rows], w, bias)
        lse = torch.logsumexp(z, 1)
        p = torch.exp(z - lse[:, None])
        far = torch.where(p > 0, (lse[:, None] - z).abs(), 0.0)
        # the largest logit's own distance from lse is at most log V; terms, their sum, its logarithm
        e = (p * (ez + (2 * far + 16) * U)).sum(1) + (80 + V / 512) * U + 2 * U * lse.abs() * torch.isfinite(lse)
        t = target[rows][:, None]
        zt = z.gather(1, t)[:, 0]
        out[0][rows], out[2][rows] = lse - zt, lse
        e = torch.nan_to_num(e, nan=0.0)
        out[1][rows] = e + ez.gather(1, t)[:, 0] + 2 * U * (lse.abs() + torch.nan_to_num(zt.abs(), posinf=0.0))
        out[3][rows] = e
    return (out[0], out[1]), (out[2], out[3])


def xent_bwd(x, w, target, lse, dloss, bias, bf16):
    """dx, dw, db as (ref, bound) from the saved lse.

    bf16: p - [target] is rounded as an operand of dx = dloss ((p - [target]) w), and with dloss x as an operand of
    dw; not for db."""
    V, K = w.shape
    half = 2.0 ** -8 if bf16 else 0.0
    rows = torch.nonzero((target >= 0) & (target < V))[:, 0]
    dx = torch.zeros(x.shape, dtype=F64, device=x.device)
    edx = torch.zeros_like(dx)
    z, ez = logits(x[rows], w, bias)
    away = z - lse.double()[rows][:, None]
    p = torch.exp(away)
    # the exponent's own error, and exp's
    ep = p * (ez + torch.where(p > 0, (3 * away.abs() + torch.nan_to_num(z.abs(), posinf=0.0) + 6) * U, 0.0))
    ep = torch.nan_to_num(ep, nan=0.0)
    dl = dloss.double()[rows][:, None]
    dz = p.clone()
    dz[torch.arange(len(rows), device=x.device), target[rows]] -= 1
    e = ep + 2 * U * dz.abs()
    op = e + dz.abs() * half
    xa, wa, n = x[rows].double(), w.double(), len(rows)
    dx[rows] = dl * (dz @ wa)
    edx[rows] = dl.abs() * ((V + 10) * U * (dz.abs() @ wa.abs()) + op @ wa.abs())
    xs = dl * xa
    t = lambda a: a.t().contiguous()  # noqa: E731
    dw = t(dz) @ xs
    edw = t((n + 8) * U * dz.abs() + op + (half + 4 * U) * (dz.abs() + op)) @ xs.abs()
    db = dl * dz
    return (dx, edx), (dw, edw), (db.sum(0), (n + 8) * U * db.abs().sum(0) + (dl.abs() * e).sum(0))


# ---- AdamW ------------------------------------------------------------------------------

def adamw(p, g, m, v, t, lr, betas, eps, decay, scale=1.0):
    """The value after a step and the new moments, as (ref, bound); p, g, m, v in any type."""
    b1, b2 = betas
    p, g, m, v = (x.double() for x in (p, g, m, v))
    g = g * scale
    mn, vn = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    # beta's and scale's roundings, two products and a sum; the square's twice
    em, ev = 4 * U * ((b1 * m).abs() + ((1 - b1) * g).abs()), 6 * U * (b2 * v + (1 - b2) * g * g)
    root = torch.sqrt(vn / (1 - b2 ** t)) + eps
    move = lr * mn / (1 - b1 ** t) / root
    # ev moves the root by half as much, in proportion
    emove = lr * em / (1 - b1 ** t) / root + move.abs() * 12 * U
    new = p * (1 - lr * decay) - move
    enew = emove + 2 * U * (p.abs() + move.abs())
    return (new, enew), (mn, em), (vn, ev)


def mix(h):
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def random_bits(n, seed, place, device):
    """The low and the high 16 bits for each element of the list's tensor ``place``."""
    i = torch.arange(n, device=device)
    h = mix((i & 0xFFFFFFFF) ^ mix((seed + 0x9E3779B9 * place + (i >> 32)) & 0xFFFFFFFF))
    return h & 0xFFFF, h >> 16


def decode(codes, scale):
    """Values of codes (float8_e4m3fn, flat) with a scale for every 256."""
    s = scale.double().repeat_interleave(256)[:codes.numel()]
    return codes.reshape(-1).double() * s


def check_codes(codes, scale, x, ex, bits, what):
    """codes and scale against the random rounding of x (flat, off by at most ex), by bits / 65536."""
    n = x.numel()
    if n == 0:
        return
    pad = torch.nn.functional.pad(x, (0, -n % 256)).view(-1, 256)
    top = pad.abs().amax(1)
    epad = torch.nn.functional.pad(ex, (0, -n % 256)).view(-1, 256).amax(1)
    check(scale, top / 448, epad / 448 + U * top / 448, what + " scale")
    s = scale.double().repeat_interleave(256)[:n]
    t = torch.where(s > 0, x.abs() / s, 0.0)
    et = torch.where(s > 0, ex / s, 0.0) + 4 * U * t
    gap = torch.exp2(torch.floor(torch.log2(t.clamp(min=2.0 ** -6))) - 3)
    place, got = t / gap, codes.reshape(-1).double().abs() / gap
    low = torch.floor(place + bits.double() / 65536)
    # where the sum lies on an integer within its error, either neighbour
    near = (place + bits.double() / 65536 - torch.round(place + bits.double() / 65536)).abs() <= et / gap + 2 * U * 16
    # (t within its error of a power of two may be counted with the finer gap's codes)
    edge = (torch.log2(t.clamp(min=2.0 ** -6)) - torch.round(torch.log2(t.clamp(min=2.0 ** -6)))).abs() < 1e-5
    fine = (got == low) | (near & ((got - low).abs() <= 1)) | (edge & ((got - low).abs() <= 1))
    assert bool(fine.all()), "%s: %d codes are not the roundings" % (what, int((~fine).sum()))
    # few may be near
    assert int((got != low).sum()) <= 4 + n * 1e-3, what
    sign = torch.where(codes.reshape(-1).double() != 0, torch.sign(codes.reshape(-1).double()) == torch.sign(x), True)
    assert bool(sign.all()), what + ": signs"
