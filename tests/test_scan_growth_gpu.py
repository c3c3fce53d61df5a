"""The gated recurrence where products of gates over a tile leave the range of fp32, against the 64-bit walk of layer_ref.

Gates above 1 (gate "log", g > 0), and small gates before large states; the
states themselves stay inside the range.  Inputs are scaled so that every output is
representable; the bounds are layer_ref's."""
import math

import numpy as np
import pytest
import torch

import gated_convolution_sequence_amd as hc
from gpu_util import DEV, log
import layer_ref as ref
from layer_ref import check, to_np
from test_scan_gpu import check_bwd, check_fwd, inputs, states_of

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    hc.layer_lib()
    yield
    torch.cuda.synchronize()


def pattern(name, L):
    """(g [L], scales of q, k, v, dy, of s0 and of ds_last; 0: no state given)."""
    t = torch.arange(L)
    if name == "two gates at the start":  # e^100 before any state is there
        g = torch.full((L,), -0.05)
        g[:2] = 50.0
        return g, (1.0, 1.0, 1.0, 1e-8), 0.0, 0.0
    if name == "up and down":  # e^96 over 64 rows, and back
        return torch.where(t // 64 % 2 == 1, 1.5, -1.5), (1e-10, 1e-12, 1e-12, 1e-10), 1e-24, 1e-20
    if name == "steep":  # e^90 over two rows, and back over the next two
        return torch.tensor([50.0, 40.0, -45.0, -45.0])[t % 4], (1e-5, 1e-15, 1e-15, 1e-5), 1e-30, 1e-10
    if name == "down and up":  # e^-224, then e^80: what is left of the state is nothing
        g = torch.full((L,), -0.1)
        g[:32], g[32:64] = -7.0, 2.5
        return g, (1e-5, 1e-15, 1e-15, 1e-5), 1e20, 1e-10
    if name == "slow":  # products stay in range
        return torch.where(t // 32 % 2 == 1, 0.25, -0.25), (1.0, 1.0, 1.0, 1.0), 1.0, 1.0
    raise ValueError(name)


PATTERNS = ("two gates at the start", "up and down", "steep", "down and up", "slow")


def make(name, B, L, D, dtype, seed):
    g, scales, first, last = pattern(name, L)
    ts = inputs(B, L, D, dtype, "log", seed)
    for i, scale in zip((0, 1, 2, 4), scales):
        ts[i].copy_(ts[i].float() * scale)
    ts[3].copy_(g[None, :, None].to(DEV))
    s0, ds_last = states_of(B, D, seed)
    return ts, (s0 * first if first else None), (ds_last * last if last else None)


@pytest.mark.parametrize("name", PATTERNS)
@pytest.mark.parametrize("B,L,D", [(1, 8, 64), (2, 63, 9), (2, 130, 64), (1, 500, 130), (2, 1000, 24)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_gates_above_one(name, B, L, D, dtype):
    log("scan growth %r %s %s" % (name, (B, L, D), dtype))
    ts, s0, ds_last = make(name, B, L, D, dtype, L + D)
    y, last, states = check_fwd(ts, "log", s0, "fwd")
    assert torch.isfinite(y).all() and torch.isfinite(last).all()
    got = check_bwd(ts, "log", s0, ds_last, states, "bwd")
    for t in got:
        assert torch.isfinite(t).all()


@pytest.mark.parametrize("D", [64, 9])
def test_one_growing_channel_among_others(D):
    """A tile with one channel out of range: the others' carries and outputs are as they should be."""
    ts, s0, ds_last = make("up and down", 2, 700, D, F32, 5)
    ts[3][:, :, torch.arange(D) != 4] = -0.3
    _, _, states = check_fwd(ts, "log", s0, "fwd")
    check_bwd(ts, "log", s0, ds_last, states, "bwd")


@pytest.mark.parametrize("name", ["up and down", "steep"])
def test_resets_infinities_and_nan_in_growing_tiles(name):
    ts, s0, ds_last = make(name, 1, 600, 72, F32, 6)
    ts[3][0, 70, 1] = math.nan
    ts[3][0, 300, :8] = -math.inf
    ts[1][0, 90, 3] = math.inf
    ts[4][0, 400, 5] = math.inf
    _, _, states = check_fwd(ts, "log", s0, "fwd")
    check_bwd(ts, "log", s0, ds_last, states, "bwd")


@pytest.mark.parametrize("name", PATTERNS)
def test_steps_agree_with_the_scan(name):
    """The same rows by scan_step, and by scan_fwd as a whole."""
    L = 140
    ts, s0, _ = make(name, 2, L, 40, F32, 8)
    y, last, _ = hc.scan_fwd(*ts[:4], gate="log", s0=s0)
    f = ref.scan_fwd(*(to_np(t) for t in ts[:4]), "log", None if s0 is None else to_np(s0))
    state = torch.zeros(2, 40, device=DEV) if s0 is None else s0.clone()
    for t in range(L):
        yt = hc.scan_step(*(x[:, t] for x in ts[:4]), state, gate="log")
        check(yt, f["y"][:, t], f["ey"][:, t], F32, "row %d" % t)
    check(last, f["last"], f["elast"], F32, "last")


def test_runs_give_the_same_bits():
    """Many growing tiles, whose carries go from state to state: run to run the same."""
    ts, s0, ds_last = make("up and down", 3, 4000, 264, BF16, 9)
    first = hc.scan_fwd(*ts[:4], gate="log", s0=s0, save_states=True)
    g1 = hc.scan_bwd(*ts, first[2], gate="log", ds_last=ds_last)
    for _ in range(4):
        for a, b in zip(hc.scan_fwd(*ts[:4], gate="log", s0=s0, save_states=True), first):
            assert torch.equal(a, b)
        for a, b in zip(hc.scan_bwd(*ts, first[2], gate="log", ds_last=ds_last), g1):
            assert torch.equal(a, b)


@pytest.mark.parametrize("gate,g", [("sigmoid", 0.0), ("log", -0.7), ("log", -3.0)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_a_large_state_under_small_gates(gate, g, dtype):
    """States and gradients of 1e30 fade over tiles whose product of gates is below fp32's least normal."""
    ts = inputs(2, 400, 40, dtype, gate, 10)
    ts[3].fill_(g)
    for i in (0, 1, 2, 4):
        ts[i].mul_(1e-8)
    s0, ds_last = states_of(2, 40, 10)
    s0, ds_last = s0 * 1e30, ds_last * 1e30
    _, _, states = check_fwd(ts, gate, s0, "fwd")
    check_bwd(ts, gate, s0, ds_last, states, "bwd")


def check_finite(got, want, bound, dtype, what):
    """As check, but what is not finite may be an infinity or NaN."""
    fin = np.isfinite(want)
    assert np.array_equal(fin, np.isfinite(to_np(got))), "%s: non-finite values differ" % what
    check(torch.where(torch.from_numpy(fin).to(DEV), got, torch.zeros_like(got)), np.where(fin, want, 0.0), bound, dtype,
          what)


@pytest.mark.parametrize("D", [64, 9])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("growing", [False, True])
@pytest.mark.parametrize("with_state", [False, True])
def test_an_infinite_gate(D, dtype, growing, with_state):
    """exp(+inf): nothing finite up to a reset, and what does not depend on it is as it should be.

    (Whether an infinity or NaN depends on the order of sums: inf (P s + S) is cut into inf s + inf.)"""
    log("scan infinite gate D=%d %s" % (D, dtype))
    ts = inputs(2, 500, D, dtype, "log", 12)
    if growing:
        ts[3].copy_(pattern("slow", 500)[0][None, :, None].to(DEV))
    s0, ds_last = states_of(2, D, 12) if with_state else (None, None)
    ts[3][0, 0, 1] = math.inf    # on the first state
    ts[3][0, 128, 2] = math.inf  # in the first row of a tile, of a slice, and inside one
    ts[3][0, 136, 3] = math.inf
    ts[3][0, 205, 4] = math.inf
    ts[3][1, 200, 5], ts[3][1, 203, 5] = math.inf, -math.inf  # a reset in the same lane's rows, and before
    ts[3][1, 201, 6], ts[3][1, 207, 6] = -math.inf, math.inf
    ts[3][1, 100, 7], ts[3][1, 300, 7] = math.inf, -math.inf
    y, last, states = hc.scan_fwd(*ts[:4], gate="log", s0=s0, save_states=True)
    a = [to_np(t) for t in ts]
    f = ref.scan_fwd(*a[:4], "log", None if s0 is None else to_np(s0))
    check_finite(last, f["last"], f["elast"], F32, "s_last")
    check_finite(states, f["states"], f["estates"], F32, "states")
    check_finite(y, f["y"], f["ey"], dtype, "y")
    want = ref.scan_bwd(*a, "log", None if s0 is None else to_np(s0), None if ds_last is None else to_np(ds_last))
    for name, t in zip(("dq", "dk", "dv", "dg", "ds0"), hc.scan_bwd(*ts, states, gate="log", ds_last=ds_last)):
        check_finite(t, *want[name], F32 if name == "ds0" else dtype, name)
