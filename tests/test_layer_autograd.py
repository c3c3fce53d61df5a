"""The autograd wrappers under create_graph=True (CPU): second derivatives raise, first ones are unchanged.

The wrappers' calls into the library are replaced by plain PyTorch forms; what
is tested is what the wrappers tell autograd."""
import pytest
import torch

import gated_convolution_sequence_amd as hc
from gated_convolution_sequence_amd import layer

F64 = torch.float64


def plain_linear_fwd(x, w, bias=None, residual=None, act="none", save_preact=False):
    z = x @ w.t() + (0 if bias is None else bias)
    y = (z * torch.sigmoid(z) if act == "silu" else z) + (0 if residual is None else residual)
    return y, z if save_preact else None


def plain_linear_bwd(x, w, dy, preact=None, act="none", need_dx=True, need_dw=True, need_db=True):
    p = torch.sigmoid(preact) if act == "silu" else None
    dz = dy * p * (1 + preact * (1 - p)) if act == "silu" else dy
    return (dz @ w if need_dx else None), (dz.t() @ x if need_dw else None), (dz.sum(0) if need_db else None)


def plain_scan_fwd(q, k, v, g, gate="sigmoid", s0=None, save_states=False):
    s, out = torch.zeros_like(q[:, 0]) if s0 is None else s0, []
    for t in range(q.shape[1]):
        s = torch.sigmoid(g[:, t]) * s + k[:, t] * v[:, t]
        out.append(s)
    s_all = torch.stack(out, 1)
    first = torch.zeros_like(q[:, :1]) if s0 is None else s0[:, None]
    return q * s_all, s, torch.cat([first, s_all[:, :-1]], 1)


def plain_scan_bwd(q, k, v, g, dy, states, gate="sigmoid", ds_last=None):
    with torch.enable_grad():
        ts = [t.detach().requires_grad_(True) for t in (q, k, v, g, states[:, 0])]
        y, last, _ = plain_scan_fwd(*ts[:4], s0=ts[4])
        return torch.autograd.grad([y, last], ts, [dy, ds_last])


@pytest.fixture(autouse=True)
def stand_ins(monkeypatch):
    for name in ("linear_fwd", "linear_bwd", "scan_fwd", "scan_bwd"):
        monkeypatch.setattr(layer, name, globals()["plain_" + name])


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F64).requires_grad_(True)


def linear_case():
    x, w, b = randn(3, 4, seed=1), randn(4, 4, seed=2), randn(4, seed=3)
    return [x, w, b], lambda x, w, b: hc.LinearAct.apply(x, w, b, x, "silu")


def scan_case():
    ts = [randn(2, 5, 3, seed=i) for i in range(4)] + [randn(2, 3, seed=9)]
    return ts, lambda q, k, v, g, s0: hc.GatedScan.apply(q, k, v, g, "sigmoid", s0)[0]


CASES = [linear_case, scan_case]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("loss", [lambda y: y.sum(), lambda y: (y * y).sum()], ids=["linear", "square"])
def test_a_second_derivative_raises(case, loss):
    """Through every input, by backward() and by grad(), with or without another way to the input beside it."""
    ts, f = case()
    for i, t in enumerate(ts):
        for beside in (False, True):
            def first():
                out = loss(f(*ts)) + ((t ** 3).sum() if beside else 0.0)
                return torch.autograd.grad(out, ts, create_graph=True)
            penalty = sum((g * g).sum() for g in first())
            with pytest.raises(RuntimeError, match="no second derivatives"):
                torch.autograd.grad(penalty, [t])
            with pytest.raises(RuntimeError, match="no second derivatives"):
                sum((g * g).sum() for g in first()).backward()


@pytest.mark.parametrize("case", CASES)
def test_first_derivatives_under_create_graph(case):
    """They are those of the plain graph, and those without create_graph."""
    ts, f = case()
    got = torch.autograd.grad((f(*ts) ** 2).sum(), ts, create_graph=True)
    plainly = torch.autograd.grad((f(*ts) ** 2).sum(), ts)
    for a, b in zip(got, plainly):
        assert torch.equal(a, b)
    if case is linear_case:
        x, w, b = ts
        want = torch.autograd.grad((plain_linear_fwd(x, w, b, x, "silu")[0] ** 2).sum(), ts)
        for a, b in zip(got, want):
            assert torch.allclose(a, b, rtol=1e-12, atol=1e-12)


def test_the_residuals_gradient_keeps_its_graph():
    """The residual's gradient is the incoming one: its second derivative is right, and does not raise."""
    x, w, r = randn(3, 4, seed=1).detach(), randn(4, 4, seed=2).detach(), randn(3, 4, seed=3)
    y = hc.LinearAct.apply(x, w, None, r, "silu")
    (g,) = torch.autograd.grad((y ** 3).sum(), [r], create_graph=True)
    (h,) = torch.autograd.grad(g.sum(), [r])
    assert torch.allclose(h, 6 * y.detach(), rtol=1e-12)
