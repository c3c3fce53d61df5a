"""The sequence-layer operators as they are measured: plain forms, the framework's calls, and their cost.

Operators (all row-major, D contiguous; bf16 or fp32 data, fp32 states):

scan    a gated linear recurrence along time,
            a_t = sigmoid(g_t) or exp(g_t),  s_t = a_t s_{t-1} + k_t v_t,  y_t = q_t s_t,
        where a_t = 0 drops the earlier state; its gradients; and its form for one token.
linear  z = x w^T + bias,  y = act(z) + residual, and its gradients.
conv    the single-token form of the gated convolution y = q (h * (k v)), with a
        ring cache of past rows of k v for each sequence.
"""
import math

import torch

own = False

DEV = "cuda:0"
CHUNK = 64  # rows between the states that the scan's forward saves for its backward


def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _eb(case):
    return 2 if case["dtype"] == "bf16" else 4


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # one sequence's next token: pure latency
        dict(name="scan_step_b1", op="scan_step", B=1, S=1, D=4096, dtype="bf16", gate="sigmoid"),
        # a large decode batch, its states scattered over a pool
        dict(name="scan_step_b256", op="scan_step", B=256, S=320, D=4096, dtype="bf16", gate="sigmoid"),
        # the medium filter's next token, one sequence
        dict(name="conv_step_b1", op="conv_step", B=1, S=1, D=4096, l_h=128, gs=16, dtype="bf16"),
        # ... and a decode batch of 64, some sequences younger than the filter
        dict(name="conv_step_b64", op="conv_step", B=64, S=80, D=4096, l_h=128, gs=16, dtype="bf16"),
        # a training forward at the framework's main size, states saved for the backward
        dict(name="scan_fwd_8k", op="scan_fwd", B=1, L=8192, D=4096, dtype="bf16", gate="sigmoid", s0=False,
             save=True, fused=False, resets=False),
        # the batched long size: a prefill of packed documents (the gate resets the
        # state), q, k, v and g being column slices of one projection's output
        dict(name="scan_fwd_b4_32k", op="scan_fwd", B=4, L=32768, D=4096, dtype="bf16", gate="sigmoid", s0=True,
             save=False, fused=True, resets=True),
        # the backward of scan_fwd_8k
        dict(name="scan_bwd_8k", op="scan_bwd", B=1, L=8192, D=4096, dtype="bf16", gate="sigmoid", s0=False,
             fused=False, resets=False),
        # fp32, ragged everywhere, a shard in the middle of a sequence (state in, gradient of the state out)
        dict(name="scan_bwd_f32_ragged", op="scan_bwd", B=3, L=1531, D=1000, dtype="f32", gate="log", s0=True,
             fused=False, resets=True),
        # the output projection of a training step: bias and residual
        dict(name="linear_fwd_8k", op="linear_fwd", M=8192, N=4096, K=4096, dtype="bf16", act="none", bias=True,
             residual=True, save=False),
        # a gate projection for the next token of 8 sequences: the weights stream once
        dict(name="linear_fwd_tokens8", op="linear_fwd", M=8, N=4096, K=4096, dtype="bf16", act="sigmoid", bias=True,
             residual=False, save=False),
        # the gradients of a projection with an activation, training step
        dict(name="linear_bwd_8k", op="linear_bwd", M=8192, N=4096, K=4096, dtype="bf16", act="silu"),
        # fp32 gradients, every size odd
        dict(name="linear_bwd_f32_odd", op="linear_bwd", M=1021, N=777, K=521, dtype="f32", act="gelu"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan_step", "conv_step", "scan_fwd", "scan_bwd", "linear_fwd", "linear_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    odd = rng.random() < 0.3
    D = _log_int(rng, 32, 4096)
    D = D | 1 if odd else max(16, D // 16 * 16)
    gate = rng.choice(["sigmoid", "log"])
    if op == "scan_step":
        B = _log_int(rng, 1, 512)
        return dict(op=op, B=B, S=B + rng.randrange(0, 64), D=D, dtype=dtype, gate=gate)
    if op == "conv_step":
        B = _log_int(rng, 1, 128)
        gs = rng.choice([g for g in (1, 2, 4, 8, 16, 32, 64) if D % g == 0])
        return dict(op=op, B=B, S=B + rng.randrange(0, 32), D=D, l_h=_log_int(rng, 1, 128), gs=gs, dtype=dtype)
    if op in ("scan_fwd", "scan_bwd"):
        L = _log_int(rng, 1, 32768)
        B = max(1, min(_log_int(rng, 1, 16), (1 << 27) // (L * D)))
        case = dict(op=op, B=B, L=L, D=D, dtype=dtype, gate=gate, s0=rng.random() < 0.5,
                    fused=rng.random() < 0.5, resets=rng.random() < 0.5)
        if op == "scan_fwd":
            case["save"] = rng.random() < 0.5
        return case
    # rows from one token to a training step's, features of either side independent
    M, N, K = _log_int(rng, 1, 8192), _log_int(rng, 64, 4096), _log_int(rng, 64, 4096)
    if not odd:
        N, K = max(16, N // 16 * 16), max(16, K // 16 * 16)
    case = dict(op=op, M=M, N=N, K=K, dtype=dtype, act=rng.choice(["none", "relu", "gelu", "silu", "sigmoid"]))
    if op == "linear_fwd":
        case.update(bias=rng.random() < 0.7, residual=rng.random() < 0.5, save=rng.random() < 0.3)
    return case


# ---- inputs ------------------------------------------------------------------

def _randn(gen, shape, dtype=torch.float32, scale=1.0):
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat, piece = out.view(-1), 1 << 27
    for s in range(0, flat.numel(), piece):
        n = min(piece, flat.numel() - s)
        flat[s:s + n].copy_(torch.randn(n, generator=gen, device=DEV).mul_(scale))
    return out


def _gates(gen, shape, case):
    """Forget gates of a trained layer: memories from a few rows to about a thousand."""
    g = _randn(gen, shape)
    if case["gate"] == "sigmoid":
        g.mul_(1.5).add_(3.5)
    else:
        g = -torch.exp(g.mul_(1.2).add_(-3.0))
    return g.to(_dt(case))


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt, st = _dt(case), dict(case)
    op = case["op"]
    if op == "scan_step":
        B, S, D = case["B"], case["S"], case["D"]
        st["slots"] = torch.randperm(S, generator=gen, device=DEV)[:B].to(torch.int32)
        # the four inputs are column slices of one projection's output
        proj = _randn(gen, (B, 4 * D), dt)
        proj[:, 3 * D:] = _gates(gen, (B, D), case)
        st["q"], st["k"], st["v"], st["g"] = (proj[:, i * D:(i + 1) * D] for i in range(4))
        st["state"] = _randn(gen, (S, D), scale=2.0)
        st["state_out"] = st["state"].clone()  # double-buffered states
    elif op == "conv_step":
        B, S, D, l_h = case["B"], case["S"], case["D"], case["l_h"]
        st["slots"] = torch.randperm(S, generator=gen, device=DEV)[:B].to(torch.int32)
        proj = _randn(gen, (B, 3 * D), dt)
        st["q"], st["k"], st["v"] = (proj[:, i * D:(i + 1) * D] for i in range(3))
        st["h"] = _randn(gen, (D // case["gs"], l_h), dt, scale=l_h ** -0.5)
        # rows in the ring: the filter's reach, rounded up
        st["cache"] = _randn(gen, (S, -(-l_h // 16) * 16, D), dt)
        # most sequences are far along; one in eight is younger than the filter
        pos = torch.randint(l_h, 100000, (B,), generator=gen, device=DEV)
        young = torch.randint(0, l_h, (B,), generator=gen, device=DEV)
        pick = torch.arange(B, device=DEV) % 8 == 5
        st["pos"] = torch.where(pick, young, pos)
    elif op in ("scan_fwd", "scan_bwd"):
        B, L, D = case["B"], case["L"], case["D"]
        if case["fused"]:
            proj = _randn(gen, (B, L, 4 * D), dt)
            q, k, v, g = (proj[:, :, i * D:(i + 1) * D] for i in range(4))
        else:
            q, k, v = (_randn(gen, (B, L, D), dt) for _ in range(3))
            g = torch.empty((B, L, D), dtype=dt, device=DEV)
        for b in range(B):
            g[b] = _gates(gen, (L, D), case)
        if case["resets"]:  # a document starts about every 2048 rows
            starts = torch.rand((B, L), generator=gen, device=DEV) < 1.0 / 2048
            g.masked_fill_(starts[:, :, None], -math.inf)
        st["q"], st["k"], st["v"], st["g"] = q, k, v, g
        st["s0_"] = _randn(gen, (B, D), scale=2.0) if case["s0"] else None
        if op == "scan_bwd":
            st["dy"] = _randn(gen, (B, L, D), dt)
            st["ds_last"] = _randn(gen, (B, D)) if case["s0"] else None
            # what the training forward saved: the state before rows 0, 64, 128, ...
            s = _scan(_decay(g, case["gate"]), k.float() * v.float(), st["s0_"])
            first = torch.zeros((B, 1, D), device=DEV) if st["s0_"] is None else st["s0_"][:, None]
            st["states"] = torch.cat([first, s[:, CHUNK - 1:L - 1:CHUNK]], dim=1).contiguous()
    else:
        M, N, K = case["M"], case["N"], case["K"]
        st["x"] = _randn(gen, (M, K), dt)
        st["w"] = _randn(gen, (N, K), dt, scale=K ** -0.5)
        if op == "linear_fwd":
            st["b"] = _randn(gen, (N,), dt, scale=0.5) if case["bias"] else None
            st["r"] = _randn(gen, (M, N), dt) if case["residual"] else None
        else:
            st["dy"] = _randn(gen, (M, N), dt)
            # what the training forward saved: z, in the data's type
            st["z"] = None if case["act"] == "none" else (st["x"].float() @ st["w"].float().t()).to(dt)
    return st


# ---- plain forms (fp32 throughout, one rounding at the end) --------------------

def _decay(g, gate):
    g = g.float()
    return torch.sigmoid(g) if gate == "sigmoid" else torch.exp(g)


def _scan(a, x, s0):
    """All states of s_t = a_t s_{t-1} + x_t along dim 1 by doubling: after the pass of
    distance n each row holds the sum over its last 2n rows (log2 L passes)."""
    s = x
    if s0 is not None:
        s = s.clone()
        s[:, 0] += a[:, 0] * s0
    n, L = 1, a.shape[1]
    while n < L:
        s = torch.cat([s[:, :n], s[:, n:] + a[:, n:] * s[:, :-n]], dim=1)
        a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], dim=1)
        n *= 2
    return s


_ACT = {
    "none": lambda z: z,
    "relu": lambda z: z.clamp(min=0),
    "gelu": lambda z: 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5))),
    "silu": lambda z: z * torch.sigmoid(z),
    "sigmoid": torch.sigmoid,
}


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    p = torch.sigmoid(z)
    return p * (1 - p)


def _plain_scan_fwd(st):
    B, L, D = st["q"].shape
    dt = st["q"].dtype
    s = _scan(_decay(st["g"], st["gate"]), st["k"].float() * st["v"].float(), st["s0_"])
    out = [(st["q"].float() * s).to(dt), s[:, -1].clone()]
    if st["save"]:
        first = torch.zeros((B, 1, D), device=s.device) if st["s0_"] is None else st["s0_"][:, None]
        out.append(torch.cat([first, s[:, CHUNK - 1:L - 1:CHUNK]], dim=1))
    return out


def _plain_scan_bwd(st):
    q, k, v, dy = (st[n].float() for n in ("q", "k", "v", "dy"))
    a = _decay(st["g"], st["gate"])
    dt = st["q"].dtype
    s = _scan(a, k * v, st["s0_"])
    first = torch.zeros_like(s[:, :1]) if st["s0_"] is None else st["s0_"][:, None]
    prev = torch.cat([first, s[:, :-1]], dim=1)
    # ds_t = q_t dy_t + a_{t+1} ds_{t+1}: the same recurrence with time turned round
    nxt = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], dim=1)
    ds = _scan(nxt.flip(1), (q * dy).flip(1), st["ds_last"]).flip(1)
    slope = torch.sigmoid(-st["g"].float()) * a if st["gate"] == "sigmoid" else a
    return [(dy * s).to(dt), (ds * v).to(dt), (ds * k).to(dt), (ds * prev * slope).to(dt), a[:, 0] * ds[:, 0]]


def _plain_scan_step(st):
    slots = st["slots"].long()
    s = _decay(st["g"], st["gate"]) * st["state"][slots] + st["k"].float() * st["v"].float()
    st["state_out"][slots] = s
    return [(st["q"].float() * s).to(st["q"].dtype), st["state_out"]]


def _plain_conv_step(st):
    cache, pos, slots, l_h = st["cache"], st["pos"], st["slots"].long(), st["l_h"]
    dt = cache.dtype
    R, D = cache.shape[1], cache.shape[2]
    x = st["k"].float() * st["v"].float()
    lag = torch.arange(1, l_h, device=pos.device)
    rows = (pos[:, None] - lag) % R
    old = cache[slots[:, None], rows].float() * (lag <= pos[:, None])[:, :, None]
    taps = st["h"].float().repeat_interleave(st["gs"], dim=0).t()  # [l_h, D]
    y = st["q"].float() * (taps[0] * x + (taps[1:] * old).sum(1))
    cache[slots, pos % R] = x.to(dt)
    return [y.to(dt), cache]


def _plain_linear_fwd(st):
    dt = st["x"].dtype
    z = st["x"].float() @ st["w"].float().t()
    if st["b"] is not None:
        z = z + st["b"].float()
    y = _ACT[st["act"]](z)
    if st["r"] is not None:
        y = y + st["r"].float()
    return [y.to(dt), z.to(dt)] if st["save"] else [y.to(dt)]


def _plain_linear_bwd(st):
    dt = st["x"].dtype
    dz = st["dy"].float()
    if st["act"] != "none":
        dz = dz * _act_grad(st["z"].float(), st["act"])
    return [(dz @ st["w"].float()).to(dt), (dz.t() @ st["x"].float()).to(dt), dz.sum(0).to(dt)]


_PLAIN = {"scan_fwd": _plain_scan_fwd, "scan_bwd": _plain_scan_bwd, "scan_step": _plain_scan_step,
          "conv_step": _plain_conv_step, "linear_fwd": _plain_linear_fwd, "linear_bwd": _plain_linear_bwd}


# ---- the framework's calls -----------------------------------------------------

def _own(st):
    import gated_convolution_sequence_amd as hc
    op = st["op"]
    if op == "scan_fwd":
        y, last, states = hc.scan_fwd(st["q"], st["k"], st["v"], st["g"], gate=st["gate"], s0=st["s0_"],
                                      save_states=st["save"])
        return [y, last, states] if st["save"] else [y, last]
    if op == "scan_bwd":
        return list(hc.scan_bwd(st["q"], st["k"], st["v"], st["g"], st["dy"], st["states"], gate=st["gate"],
                                ds_last=st["ds_last"]))
    if op == "scan_step":
        y = hc.scan_step(st["q"], st["k"], st["v"], st["g"], st["state"], slots=st["slots"], gate=st["gate"],
                         state_out=st["state_out"])
        return [y, st["state_out"]]
    if op == "conv_step":
        y = hc.conv_step(st["q"], st["k"], st["v"], st["h"], st["cache"], st["pos"], st["gs"], slots=st["slots"])
        return [y, st["cache"]]
    if op == "linear_fwd":
        y, z = hc.linear_fwd(st["x"], st["w"], bias=st["b"], residual=st["r"], act=st["act"],
                             save_preact=st["save"])
        return [y, z] if st["save"] else [y]
    return list(hc.linear_bwd(st["x"], st["w"], st["dy"], preact=st["z"], act=st["act"]))


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ---- the definition in 64 bits ---------------------------------------------------

def _to_double(state, names):
    return [None if state.get(n) is None else state[n].double() for n in names]


def _exact_scan(state):
    """Row by row, as the recurrence is written."""
    back = state["op"] == "scan_bwd"
    B, L, D = state["q"].shape

    def row(name, t):
        return state[name][:, t].double()

    def gate(t):
        g = row("g", t)
        return 1 / (1 + torch.exp(-g)) if state["gate"] == "sigmoid" else torch.exp(g)

    zero = torch.zeros((B, D), dtype=torch.float64, device=state["q"].device)
    s = zero if state["s0_"] is None else state["s0_"].double()
    kept = torch.empty((L + 1, B, D), dtype=torch.float64, device=s.device) if back else None
    y, saved = ([] if back else torch.empty((B, L, D), dtype=torch.float64, device=s.device)), []
    for t in range(L):
        if t % CHUNK == 0:
            saved.append(s)
        if back:
            kept[t] = s
        s = gate(t) * s + row("k", t) * row("v", t)
        if not back:
            y[:, t] = row("q", t) * s
    if not back:
        return [y, s, torch.stack(saved, dim=1)] if state["save"] else [y, s]
    kept[L] = s
    c = zero if state["ds_last"] is None else state["ds_last"].double()
    out = [torch.empty((B, L, D), dtype=torch.float64, device=s.device) for _ in range(4)]
    for t in reversed(range(L)):
        ds, a, dy = row("q", t) * row("dy", t) + c, gate(t), row("dy", t)
        out[0][:, t] = dy * kept[t + 1]
        out[1][:, t] = ds * row("v", t)
        out[2][:, t] = ds * row("k", t)
        out[3][:, t] = ds * kept[t] * (a * (1 - a) if state["gate"] == "sigmoid" else a)
        c = a * ds
    return out + [c]


def _exact_linear(state):
    act = state["act"]

    def phi(z):
        return 0.5 * torch.erfc(-z / math.sqrt(2.0))

    x, w = state["x"].double(), state["w"].double()
    if state["op"] == "linear_fwd":
        z = torch.nn.functional.linear(x, w, None if state["b"] is None else state["b"].double())
        y = {"none": lambda: z, "relu": lambda: torch.where(z > 0, z, torch.zeros_like(z)),
             "gelu": lambda: z * phi(z), "silu": lambda: z / (1 + torch.exp(-z)),
             "sigmoid": lambda: 1 / (1 + torch.exp(-z))}[act]()
        if state["r"] is not None:
            y = y + state["r"].double()
        return [y, z] if state["save"] else [y]
    dz = state["dy"].double()
    if act != "none":
        z = state["z"].double()
        e = torch.exp(-z)
        dz = dz * {"relu": lambda: torch.where(z > 0, 1.0, 0.0).double(),
                   "gelu": lambda: phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi),
                   "silu": lambda: (1 + e + z * e) / (1 + e) ** 2,
                   "sigmoid": lambda: e / (1 + e) ** 2}[act]()
    return [dz @ w, dz.t() @ x, dz.sum(0)]


def exact(case, seed):
    if case["op"] in ("scan_fwd", "scan_bwd") and case["B"] * case["L"] * case["D"] > (1 << 30):
        return None
    state = prepare(case, seed)
    if case["op"] in ("scan_fwd", "scan_bwd"):
        return _exact_scan(state)
    if case["op"].startswith("linear"):
        return _exact_linear(state)
    slots = state["slots"].long()
    q, k, v = _to_double(state, ("q", "k", "v"))
    if case["op"] == "scan_step":
        g = state["g"].double()
        a = torch.exp(g) if case["gate"] == "log" else torch.exp(-torch.log1p(torch.exp(-g)))
        s = k * v + a * state["state"].double().index_select(0, slots)
        whole = state["state_out"].double().index_copy(0, slots, s)
        return [q * s, whole]
    # conv_step: tap by tap
    cache, pos, h, gs = state["cache"].double(), state["pos"], state["h"].double(), case["gs"]
    R = cache.shape[1]
    filt = torch.arange(case["D"], device=pos.device) // gs
    total = h[filt, 0] * (k * v)
    for s in range(1, case["l_h"]):
        past = cache[slots, torch.remainder(pos - s, R)]
        total = total + torch.where((pos >= s)[:, None], h[filt, s] * past, torch.zeros_like(past))
    cache[slots, torch.remainder(pos, R)] = k * v
    return [q * total, cache]


# ---- what a pass cannot do without -------------------------------------------------

def work(case):
    op, eb = case["op"], _eb(case)
    if op == "scan_step":
        n = case["B"] * case["D"]
        return {"bytes": n * (5 * eb + 8) + 4 * case["B"], "flops": 8 * n}
    if op == "conv_step":
        n = case["B"] * case["D"]
        # one sequence in eight is on average half a filter old
        rows = case["l_h"] - 1
        return {"bytes": n * eb * (rows + 5) + case["D"] // case["gs"] * case["l_h"] * eb + 12 * case["B"],
                "flops": n * (2 * case["l_h"] + 2)}
    if op in ("scan_fwd", "scan_bwd"):
        B, L, D = case["B"], case["L"], case["D"]
        n, chunks = B * L * D, B * -(-L // CHUNK) * D
        if op == "scan_fwd":
            return {"bytes": 5 * n * eb + 4 * B * D * (2 if case["s0"] else 1) + (4 * chunks if case["save"] else 0),
                    "flops": 8 * n}
        return {"bytes": 9 * n * eb + 4 * B * D * (2 if case["s0"] else 1) + 4 * chunks, "flops": 18 * n}
    M, N, K = case["M"], case["N"], case["K"]
    if op == "linear_fwd":
        wide = M * N * (1 + case["residual"] + case["save"])
        return {"bytes": eb * (M * K + N * K + wide + (N if case["bias"] else 0)), "flops": 2 * M * N * K + 4 * M * N}
    return {"bytes": eb * (2 * M * K + 2 * N * K + M * N * (1 if case["act"] == "none" else 2) + N),
            "flops": 4 * M * N * K + 4 * M * N}
