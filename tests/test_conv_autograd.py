"""HyenaConv and HyenaConvLong under create_graph=True (CPU): second derivatives raise, first ones are unchanged.

The library's calls are replaced by plain PyTorch forms."""
import pytest
import torch

import gated_convolution_sequence_amd as hc

F64 = torch.float64


def plain_fwd(q, k, v, h, group_size, workspace=None):
    x, taps = k * v, h.repeat_interleave(group_size, dim=0).t()
    L = q.shape[1]
    out = sum(taps[s] * torch.cat([torch.zeros_like(x[:, :s]), x[:, :L - s]], 1) for s in range(min(L, h.shape[1])))
    return q * out


def plain_bwd(q, k, v, h, dy, group_size, need_dq=True, need_dkv=True, need_dh=True, **_):
    with torch.enable_grad():
        ts = [t.detach().requires_grad_(True) for t in (q, k, v, h)]
        grads = torch.autograd.grad(plain_fwd(*ts, group_size), ts, dy)
    return tuple(g if n else None for g, n in zip(grads, (need_dq, need_dkv, need_dkv, need_dh)))


@pytest.fixture(autouse=True)
def stand_ins(monkeypatch):
    monkeypatch.setattr(hc, "conv_fwd", plain_fwd)
    monkeypatch.setattr(hc, "conv_fwd_long", plain_fwd)
    monkeypatch.setattr(hc, "conv_bwd", plain_bwd)
    monkeypatch.setattr(hc, "conv_bwd_long", plain_bwd)
    monkeypatch.setattr(hc, "bwd_long_workspace_bytes", lambda *a: 16)
    monkeypatch.setattr(hc, "_dtype_code", lambda dt: 0)


def tensors(l_h):
    gen = torch.Generator().manual_seed(l_h)
    mk = lambda *s: torch.randn(*s, generator=gen, dtype=F64).requires_grad_(True)  # noqa: E731
    return [mk(2, 6, 4), mk(2, 6, 4), mk(2, 6, 4), mk(2, l_h)]


@pytest.mark.parametrize("fn,l_h", [(hc.HyenaConv, 3), (hc.HyenaConv, 130), (hc.HyenaConvLong, 3)])
def test_a_second_derivative_raises(fn, l_h):
    ts = tensors(l_h)
    want = torch.autograd.grad((plain_fwd(*ts, 2) ** 2).sum(), ts)
    for a, b in zip(torch.autograd.grad((fn.apply(*ts, 2) ** 2).sum(), ts, create_graph=True), want):
        assert torch.allclose(a, b, rtol=1e-12, atol=1e-12)
    for t in ts:
        for beside in (False, True):
            out = (fn.apply(*ts, 2) ** 2).sum() + ((t ** 3).sum() if beside else 0.0)
            penalty = sum((g * g).sum() for g in torch.autograd.grad(out, ts, create_graph=True))
            with pytest.raises(RuntimeError, match="no second derivatives"):
                torch.autograd.grad(penalty, [t])
