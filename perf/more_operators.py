"""The operators between a model's layers and its weights as they are measured: plain forms, the framework's calls, cost.

Operators (rows are contiguous; bf16 or fp32 data, fp32 statistics, losses and optimizer states):

norm    y = (x - mean) rstd w + b over a row's D channels (kind "layer"), or
        y = x rstd w + b with the root mean square (kind "rms"); its gradients.
xent    the softmax cross entropy of a readout, z = x w^T + bias over a vocabulary,
            lse_i = log sum_v exp(z_iv),   loss_i = lse_i - z_i,target_i
        (0 where the target is no entry of the vocabulary), and the gradients of x, w and bias.
adamw   the clipping scale of all gradients together and one AdamW step over a list of tensors,
        the moments in fp32, or m and sqrt(v) in 8 bits (e4m3) with a scale for every 256, rounded
        up or down at random in proportion.
"""
import math

import torch

own = False

DEV = "cuda:0"
EPS = 1e-5
BETAS, ADAM_EPS, DECAY = (0.9, 0.95), 1e-8, 0.1


def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _eb(case):
    return 2 if case["dtype"] == "bf16" else 4


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # the norm before a layer, one sequence's next token: pure latency
        dict(name="norm_fwd_token", op="norm_fwd", M=1, D=4096, dtype="bf16", kind="layer", strided=False),
        # ... in a training forward at the framework's main size
        dict(name="norm_fwd_8k", op="norm_fwd", M=8192, D=4096, dtype="bf16", kind="layer", strided=False),
        # ... and its backward
        dict(name="norm_bwd_8k", op="norm_bwd", M=8192, D=4096, dtype="bf16", kind="layer", strided=False),
        # fp32, odd sizes, x a column slice of a wider buffer, root mean square
        dict(name="norm_bwd_f32_ragged", op="norm_bwd", M=4593, D=1001, dtype="f32", kind="rms", strided=True),
        # the scores of a few positions under a large vocabulary: the weights stream once
        dict(name="xent_fwd_rows8", op="xent_fwd", M=8, K=4096, V=65536, dtype="bf16", bias=False, masked=0.0),
        # a training step's loss
        dict(name="xent_fwd_8k", op="xent_fwd", M=8192, K=4096, V=65536, dtype="bf16", bias=False, masked=0.0),
        # ... and its gradients, a quarter of the positions being prompt or padding without a target
        dict(name="xent_bwd_8k", op="xent_bwd", M=8192, K=4096, V=65536, dtype="bf16", bias=False, masked=0.25),
        # a byte-level vocabulary: as many rows, few columns
        dict(name="xent_bwd_bytes", op="xent_bwd", M=8192, K=4096, V=512, dtype="bf16", bias=True, masked=0.0),
        # fp32, every size odd
        dict(name="xent_bwd_f32_odd", op="xent_bwd", M=1021, K=777, V=5003, dtype="f32", bias=True, masked=0.3),
        # the example model's weights at width 256: launches count
        dict(name="adamw_small", op="adamw", D=256, V=32, layers=1, dtype="bf16", master=True, clip=True, bits=32),
        # a layer of the main width and a large embedding, fp32 masters of bf16 weights
        dict(name="adamw_large", op="adamw", D=4096, V=65536, layers=1, dtype="bf16", master=True, clip=True, bits=32),
        # the moments in 8 bits
        dict(name="adamw_8bit", op="adamw", D=4096, V=512, layers=2, dtype="bf16", master=True, clip=True, bits=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "xent_fwd", "xent_bwd", "adamw"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    odd = rng.random() < 0.3
    if op in ("norm_fwd", "norm_bwd"):
        D = _log_int(rng, 32, 8192)
        D = D | 1 if odd else max(16, D // 16 * 16)
        M = min(_log_int(rng, 1, 32768), (1 << 26) // D)
        return dict(op=op, M=M, D=D, dtype=dtype, kind=rng.choice(["layer", "rms"]), strided=rng.random() < 0.3)
    if op in ("xent_fwd", "xent_bwd"):
        M, K, V = _log_int(rng, 1, 8192), _log_int(rng, 64, 4096), _log_int(rng, 4, 65536)
        if not odd:
            K = max(16, K // 16 * 16)
        if dtype == "f32":  # fp32 products are slower by the card's rates
            V = max(4, min(V, (1 << 37) // (M * K)))
        return dict(op=op, M=M, K=K, V=V, dtype=dtype, bias=rng.random() < 0.4,
                    masked=rng.choice([0.0, 0.0, 0.1, 0.5, 0.9]))
    D = _log_int(rng, 32, 2048)
    D = D | 1 if odd else max(16, D // 16 * 16)
    return dict(op=op, D=D, V=_log_int(rng, 16, 32768), layers=rng.randrange(1, 5), dtype=dtype,
                master=dtype == "bf16" and rng.random() < 0.7, clip=rng.random() < 0.7, bits=rng.choice([32, 32, 8]))


def _active(case):
    """Rows with a target."""
    return case["M"] - int(case["M"] * case["masked"])


def _shapes(case):
    """The weights of a model: an embedding, a readout, and per layer two mixers with their projections and norms."""
    D, shapes = case["D"], [(case["V"], case["D"])] * 2
    for _ in range(case["layers"]):
        shapes += [(D,)] * 4 + [(D, D)] * 4 + [(max(1, D // 16), 128)] + [(4 * D, D), (4 * D,), (D, D)]
    return shapes


BLOCK = 256  # elements that share a scale where the moments have 8 bits


def _room(shape, unit=BLOCK):
    return -(-math.prod(shape) // unit) * unit


def _views(flat, shapes, unit=BLOCK):
    out, at = [], 0
    for sh in shapes:
        out.append(flat[at:at + math.prod(sh)].view(sh))
        at += _room(sh, unit)
    return out


# ---- inputs ------------------------------------------------------------------

def _randn(gen, shape, dtype=torch.float32, scale=1.0):
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat, piece = out.view(-1), 1 << 27
    for s in range(0, flat.numel(), piece):
        n = min(piece, flat.numel() - s)
        flat[s:s + n].copy_(torch.randn(n, generator=gen, device=DEV).mul_(scale))
    return out


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt, st = _dt(case), dict(case)
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        M, D = case["M"], case["D"]
        # a residual stream: channels of unlike size and mean
        x = _randn(gen, (M, 2 * D if case["strided"] else D))
        x.mul_(1 + _randn(gen, (x.shape[1],)).abs()).add_(_randn(gen, (x.shape[1],), scale=0.5))
        st["x"] = x.to(dt)[:, :D]
        st["w"] = (1 + _randn(gen, (D,), scale=0.2)).to(dt)
        st["b"] = _randn(gen, (D,), dt, scale=0.2) if case["kind"] == "layer" else None
        if op == "norm_bwd":
            st["dy"] = _randn(gen, (M, D), dt)
            # what the training forward saved
            mean, rstd = _stats(st["x"].double(), case["kind"])
            st["mean"], st["rstd"] = None if mean is None else mean.float(), rstd.float()
    elif op in ("xent_fwd", "xent_bwd"):
        M, K, V = case["M"], case["K"], case["V"]
        st["x"] = _randn(gen, (M, K), dt)  # behind the last norm
        st["w"] = _randn(gen, (V, K), dt, scale=2 * K ** -0.5)
        st["b"] = _randn(gen, (V,), dt, scale=0.5) if case["bias"] else None
        # few tokens are frequent, most are rare
        target = (torch.rand(M, generator=gen, device=DEV, dtype=torch.float64) ** 3 * V).long().clamp_(max=V - 1)
        target[torch.randperm(M, generator=gen, device=DEV)[:M - _active(case)]] = -100
        st["target"] = target
        if op == "xent_bwd":
            # the mean over the rows with a target, each weighted
            st["dloss"] = (0.5 + torch.rand(M, generator=gen, device=DEV)) / max(1, _active(case))
            # what the training forward saved
            st["lse"] = torch.where(target >= 0, torch.logsumexp(_logits(st), dim=1), 0.0)
    else:
        # the lists are views of one buffer each, tensors at multiples of 256 elements
        shapes = _shapes(case)
        flat = _randn(gen, (sum(_room(sh) for sh in shapes),))
        for t, sh in zip(_views(flat, shapes), shapes):
            t.mul_(sh[-1] ** -0.5 if len(sh) == 2 else 1.0)
        st["params_flat"] = flat.to(dt)
        st["masters_flat"] = flat if case["master"] else None
        st["grads"] = _views(_randn(gen, flat.shape, dt, scale=1e-3), shapes)
        # moments some way into a training
        st["m_flat"] = _randn(gen, flat.shape, scale=5e-4)
        st["v_flat"] = _randn(gen, flat.shape, scale=1e-3).square_()
        if case["bits"] == 8:
            st["v_flat"].sqrt_()
            for n in "mv":
                scale = st[n + "_flat"].view(-1, BLOCK).abs().amax(1) / 448
                codes = (st[n + "_flat"].view(-1, BLOCK) / scale[:, None]).to(torch.float8_e4m3fn)
                st[n + "_flat"], st[n + "_scale_flat"] = codes.view(-1), scale
                st[n + "_scale"] = _views(scale, [(-(-math.prod(sh) // BLOCK),) for sh in shapes], 1)
        for n, key in (("params", "params_flat"), ("masters", "masters_flat"), ("m", "m_flat"), ("v", "v_flat")):
            st[n] = None if st[key] is None else _views(st[key], shapes)
        st["step"], st["lr"], st["seed"] = 1000, 3e-4, 20240
    return st


# ---- plain forms (fp32 throughout, one rounding at the end) --------------------

def _stats(x, kind):
    """Mean and reciprocal deviation of each row (kind "rms": no mean)."""
    mean = x.mean(1) if kind == "layer" else None
    d = x if mean is None else x - mean[:, None]
    return mean, 1 / torch.sqrt((d * d).mean(1) + EPS)


def _plain_norm_fwd(st):
    x = st["x"].float()
    mean, rstd = _stats(x, st["kind"])
    y = (x if mean is None else x - mean[:, None]) * rstd[:, None] * st["w"].float()
    if st["b"] is not None:
        y = y + st["b"].float()
    return [y.to(st["x"].dtype)] + ([] if mean is None else [mean]) + [rstd]


def _plain_norm_bwd(st):
    x, dy, w, rstd = st["x"].float(), st["dy"].float(), st["w"].float(), st["rstd"][:, None]
    dt = st["x"].dtype
    unit = (x if st["mean"] is None else x - st["mean"][:, None]) * rstd
    g = dy * w
    dx = g - unit * (g * unit).mean(1, keepdim=True)
    if st["mean"] is not None:
        dx = dx - g.mean(1, keepdim=True)
    out = [(dx * rstd).to(dt), (dy * unit).sum(0).to(dt)]
    return out + ([dy.sum(0).to(dt)] if st["b"] is not None else [])


def _logits(st):
    z = st["x"].float() @ st["w"].float().t()
    return z if st["b"] is None else z + st["b"].float()


def _plain_xent_fwd(st):
    z, target = _logits(st), st["target"]
    top = z.max(1, keepdim=True).values
    lse = (top + torch.log(torch.exp(z - top).sum(1, keepdim=True)))[:, 0]
    at = z.gather(1, target.clamp(min=0)[:, None])[:, 0]
    return [torch.where(target >= 0, lse - at, 0.0), torch.where(target >= 0, lse, 0.0)]


def _plain_xent_bwd(st):
    dt, target = st["x"].dtype, st["target"]
    dz = torch.exp(_logits(st) - st["lse"][:, None])
    dz.scatter_add_(1, target.clamp(min=0)[:, None], -torch.ones_like(dz[:, :1]))
    dz *= torch.where(target >= 0, st["dloss"], 0.0)[:, None]
    out = [(dz @ st["w"].float()).to(dt), (dz.t() @ st["x"].float()).to(dt)]
    return out + ([dz.sum(0).to(dt)] if st["b"] is not None else [])


def _adamw_outputs(st, norm):
    names = ["params", "m", "v"] + (["masters"] if st["masters"] else [])
    names += ["m_scale", "v_scale"] if st["bits"] == 8 else []
    return [st[n + "_flat"] for n in names] + ([] if norm is None else [norm])


def _mix(h):
    """32 bits well mixed (the last steps of murmur3)."""
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _random_bits(n, seed, tensor):
    """Two times 16 bits for each of n elements of a tensor: those of m and of v."""
    i = torch.arange(n, device=DEV)
    key = _mix((seed + tensor * 0x9E3779B9 + (i >> 32)) & 0xFFFFFFFF)
    h = _mix((i & 0xFFFFFFFF) ^ key)
    return h & 0xFFFF, h >> 16


def _to_codes(x, bits):
    """e4m3 codes and scales of x's blocks, each rounded up with the probability of its place between two codes."""
    n = x.numel()
    x = torch.nn.functional.pad(x.view(-1), (0, -n % BLOCK)).view(-1, BLOCK)
    scale = x.abs().amax(1) / 448
    t = torch.where(scale[:, None] > 0, x.abs() / scale[:, None], 0.0).clamp(max=448)
    exponent = torch.frexp(t).exponent - 1
    step = torch.ldexp(torch.ones_like(t), exponent.clamp(min=-6) - 3)
    up = torch.nn.functional.pad(bits, (0, -n % BLOCK)).view(-1, BLOCK).float() / 65536
    q = torch.floor(t / step + up) * step
    return torch.copysign(q, x).view(-1)[:n].to(torch.float8_e4m3fn), scale


def _from_codes(codes, scale):
    n = codes.numel()
    return codes.view(-1).float() * scale.repeat_interleave(BLOCK)[:n]


def _plain_adamw(st):
    (b1, b2), lr, t = BETAS, st["lr"], st["step"]
    grads = [g.float() for g in st["grads"]]
    norm, scale = None, 1.0
    if st["clip"]:
        norm = torch.sqrt(torch.stack([(g * g).sum() for g in grads]).sum())
        scale = torch.clamp(1.0 / norm, max=1.0)
    # one tensor at a time, since each has a size of its own
    for i, g in enumerate(grads):
        g = g * scale
        m, v = st["m"][i], st["v"][i]
        if st["bits"] == 8:
            m = _from_codes(m, st["m_scale"][i]).view(g.shape)
            v = _from_codes(v, st["v_scale"][i]).square().view(g.shape)
        m = m * b1 + g * (1 - b1)
        v = v * b2 + g * g * (1 - b2)
        value = st["masters"][i] if st["masters"] else st["params"][i].float()
        move = m / (1 - b1 ** t) / (torch.sqrt(v / (1 - b2 ** t)) + ADAM_EPS)
        value = value * (1 - lr * DECAY) - lr * move
        if st["masters"]:
            st["masters"][i].copy_(value)
        st["params"][i].copy_(value)
        if st["bits"] == 8:
            for name, x, bits in zip("mv", (m, v.sqrt()), _random_bits(g.numel(), st["seed"], i)):
                codes, scales = _to_codes(x, bits)
                st[name][i].copy_(codes.view(g.shape))
                st[name + "_scale"][i].copy_(scales)
        else:
            st["m"][i].copy_(m)
            st["v"][i].copy_(v)
    return _adamw_outputs(st, norm)


_PLAIN = {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "xent_fwd": _plain_xent_fwd,
          "xent_bwd": _plain_xent_bwd, "adamw": _plain_adamw}


# ---- the framework's calls -----------------------------------------------------

def _own(st):
    import gated_convolution_sequence_amd as hc
    op = st["op"]
    if op == "norm_fwd":
        y, mean, rstd = hc.norm_fwd(st["x"], st["w"], st["b"], kind=st["kind"], eps=EPS, save_stats=True)
        return [y] + ([] if mean is None else [mean]) + [rstd]
    if op == "norm_bwd":
        got = hc.norm_bwd(st["x"], st["w"], st["dy"], st["mean"], st["rstd"], kind=st["kind"],
                          need_db=st["b"] is not None)
        return [t for t in got if t is not None]
    if op == "xent_fwd":
        return list(hc.xent_fwd(st["x"], st["w"], st["target"], bias=st["b"]))
    if op == "xent_bwd":
        got = hc.xent_bwd(st["x"], st["w"], st["target"], st["lse"], st["dloss"], bias=st["b"],
                          need_db=st["b"] is not None)
        return [t for t in got if t is not None]
    norm = scale = None
    if st["clip"]:
        norm, scale = hc.grad_norm(st["grads"], max_norm=1.0)
    hc.adamw_step(st["params"], st["grads"], st["m"], st["v"], step=st["step"], lr=st["lr"], betas=BETAS,
                  eps=ADAM_EPS, weight_decay=DECAY, masters=st["masters"], grad_scale=scale,
                  exp_avg_scales=st.get("m_scale"), exp_avg_sq_scales=st.get("v_scale"), seed=st["seed"])
    return _adamw_outputs(st, norm)


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ---- the definition in 64 bits ---------------------------------------------------

def _exact_norm(st):
    x, w = st["x"].double(), st["w"].double()
    rms = st["kind"] == "rms"
    if st["op"] == "norm_fwd":
        centre = torch.zeros_like(x[:, :1]) if rms else x.sum(1, keepdim=True) / x.shape[1]
        r = ((x - centre).pow(2).sum(1, keepdim=True) / x.shape[1] + EPS).pow(-0.5)
        y = torch.addcmul(torch.zeros_like(w) if st["b"] is None else st["b"].double(), (x - centre) * r, w)
        return [y] + ([] if rms else [centre[:, 0]]) + [r[:, 0]]
    # dx is what remains of g = w dy, without its parts along 1 (not for rms) and along the normed row
    dy, r = st["dy"].double(), st["rstd"].double()
    u = x * r[:, None] if rms else (x - st["mean"].double()[:, None]) * r[:, None]
    g = w * dy
    dots = torch.einsum("md,md->m", g, u) / x.shape[1]
    dx = g - torch.einsum("m,md->md", dots, u)
    if not rms:
        dx = dx - (g.sum(1) / x.shape[1])[:, None]
    out = [torch.einsum("md,m->md", dx, r), torch.einsum("md,md->d", dy, u)]
    return out + ([torch.einsum("md->d", dy)] if st["b"] is not None else [])


def _exact_xent(st):
    x, w, target = st["x"].double(), st["w"].double(), st["target"]
    rows = torch.nonzero(target >= 0)[:, 0]
    z = torch.nn.functional.linear(x[rows], w, None if st["b"] is None else st["b"].double())
    t, here = target[rows], torch.arange(len(rows), device=z.device)
    if st["op"] == "xent_fwd":
        lse = torch.logsumexp(z, dim=1)
        out = [torch.zeros(len(target), dtype=torch.float64, device=z.device) for _ in range(2)]
        out[0][rows], out[1][rows] = lse - z[here, t], lse
        return out
    p = z.sub_(st["lse"].double()[rows, None]).exp_()
    p[here, t] -= 1.0
    p *= st["dloss"].double()[rows, None]
    dx = torch.zeros_like(x)
    dx[rows] = torch.matmul(p, w)
    out = [dx, torch.matmul(p.t(), x[rows])]
    return out + ([p.sum(0)] if st["b"] is not None else [])


def _exact_codes(x, chance):
    """The e4m3 values between which each x / scale lies are 2^k apart; up or down by chance."""
    scale = torch.nn.functional.pad(x, (0, -len(x) % BLOCK)).view(-1, BLOCK).abs().amax(1) / 448
    t = x / scale.repeat_interleave(BLOCK)[:len(x)]
    t = torch.nan_to_num(t, nan=0.0)
    gap = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
    low = torch.floor(t.abs() / gap)
    return torch.sign(t) * (low + (t.abs() / gap - low + chance >= 1)) * gap, scale


def _exact_adamw(st):
    (b1, b2), lr, t = BETAS, st["lr"], st["step"]
    norm, scale = None, 1.0
    if st["clip"]:
        norm = math.sqrt(sum(float(g.double().pow(2).sum()) for g in st["grads"]))
        scale = min(1.0, 1.0 / norm)
    names = ["params", "m", "v"] + (["masters"] if st["masters"] else [])
    names += ["m_scale", "v_scale"] if st["bits"] == 8 else []
    flat = {n: st[n + "_flat"].double() for n in names}
    shapes = [g.shape for g in st["grads"]]
    out = {n: _views(flat[n], shapes) for n in names if "scale" not in n}
    for i, g in enumerate(st["grads"]):
        g = g.double() * scale
        m, v = out["m"][i], out["v"][i]
        if st["bits"] == 8:
            m, v = ((c.view(-1) * s[i].double().repeat_interleave(BLOCK)[:c.numel()]).view(g.shape)
                    for c, s in ((m, st["m_scale"]), (v, st["v_scale"])))
            v = v ** 2
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g ** 2
        p = (st["masters"] or st["params"])[i].double()
        p = p - lr * DECAY * p - lr * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)) ** 0.5 + ADAM_EPS)
        out["params"][i].copy_(p)
        if st["masters"]:
            out["masters"][i].copy_(p)
        if st["bits"] == 8:
            for n, x, bits in zip("mv", (m, v ** 0.5), _random_bits(g.numel(), st["seed"], i)):
                codes, scales = _exact_codes(x.reshape(-1), bits.double() / 65536)
                out[n][i].copy_(codes.view(g.shape))
                at = st[n + "_scale"][i].storage_offset()
                flat[n + "_scale"][at:at + len(scales)] = scales
        else:
            out["m"][i].copy_(m)
            out["v"][i].copy_(v)
    return [flat[n] for n in names] + ([] if norm is None else [torch.tensor(norm, dtype=torch.float64, device=DEV)])


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(state)
    return _exact_xent(state) if case["op"].startswith("xent") else _exact_adamw(state)


# ---- what a pass cannot do without -------------------------------------------------

def work(case):
    op, eb = case["op"], _eb(case)
    if op in ("norm_fwd", "norm_bwd"):
        n, M, D = case["M"] * case["D"], case["M"], case["D"]
        layer = case["kind"] == "layer"
        if op == "norm_fwd":
            return {"bytes": 2 * n * eb + D * eb * (1 + layer) + 4 * M * (1 + layer), "flops": 8 * n}
        return {"bytes": 3 * n * eb + D * eb * (2 + layer) + 4 * M * (1 + layer), "flops": 14 * n}
    if op in ("xent_fwd", "xent_bwd"):
        M, K, V, rows = case["M"], case["K"], case["V"], _active(case)
        bias = V * eb if case["bias"] else 0
        if op == "xent_fwd":
            return {"bytes": eb * (rows * K + V * K) + bias + 16 * M, "flops": 2 * rows * K * V + 4 * rows * V}
        # the logits are not kept: they are formed again, before the two products of the gradients
        return {"bytes": eb * (rows * K + M * K + 2 * V * K) + 2 * bias + 16 * M,
                "flops": 6 * rows * K * V + 4 * rows * V}
    n = sum(math.prod(s) for s in _shapes(case))
    # gradient in, parameter out (and in, without a master); master, and the moments, both ways
    each = 2 * eb + (8 if case["master"] else eb) + (16 if case["bits"] == 32 else 4 + 16 / BLOCK)
    return {"bytes": int(n * each), "flops": n * (14 + (2 if case["clip"] else 0) + (10 if case["bits"] == 8 else 0))}
