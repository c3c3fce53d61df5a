"""The example model of examples/sequence_layers.py: gradients, training, and decoding against the full forward."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import gated_convolution_sequence_amd as hc
from gpu_util import DEV, log

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("sequence_layers", os.path.join(ROOT, "examples", "sequence_layers.py"))
ex = importlib.util.module_from_spec(spec)
spec.loader.exec_module(ex)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    hc.layer_lib()
    hc.lib()
    yield
    torch.cuda.synchronize()


def plain_forward(model, tokens):
    """The model in 64 bits on the CPU, from the operators' definitions; differentiable."""
    p = {n: v.detach().cpu().double().requires_grad_(True) for n, v in model.named_parameters()}
    D, L = model.width, tokens.shape[1]
    x = p["embed"][tokens]
    q, k, v = (x @ p["conv_in.%d" % i].t() for i in range(3))
    taps = p["taps"].repeat_interleave(ex.GROUP, dim=0)
    u = k * v
    conv = torch.zeros_like(u)
    for s in range(min(ex.TAPS, L)):
        conv = conv + torch.cat([torch.zeros_like(u[:, :s]), taps[:, s] * u[:, :L - s]], dim=1)
    x = x + (q * conv) @ p["conv_out"].t()
    z = x @ p["scan_in"].t() + p["scan_bias"]
    q, k, v, g = (z[..., i * D:(i + 1) * D] for i in range(4))
    s, rows = torch.zeros_like(q[:, 0]), []
    for t in range(L):
        s = torch.sigmoid(g[:, t]) * s + k[:, t] * v[:, t]
        rows.append(q[:, t] * s)
    x = x + torch.stack(rows, dim=1) @ p["scan_out"].t()
    return x @ p["readout"].t(), p


def test_gradients_of_the_whole_model():
    """fp32 model against 64 bits: every parameter's gradient.  Each is a sum of some thousands of products
    through a dozen fp32 operators: 2^-14 of its largest element."""
    model = ex.Model(64, dtype=torch.float32)
    tokens = ex.batch(3, 21, torch.Generator().manual_seed(5))
    weight = torch.randn(3, 42, ex.VOCAB, generator=torch.Generator().manual_seed(6))
    got = model(tokens.to(DEV))
    (got * weight.to(DEV)).sum().backward()
    want, p = plain_forward(model, tokens)
    (want * weight.double()).sum().backward()
    assert (got.detach().cpu().double() - want).abs().max() <= 2.0 ** -14 * want.abs().max()
    for name, v in model.named_parameters():
        err = (v.grad.cpu().double() - p[name].grad).abs().max()
        assert err <= 2.0 ** -14 * p[name].grad.abs().max(), (name, err)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("prompt", [1, 5, 30])
def test_decoding_follows_the_forward(dtype, prompt):
    """A prompt in one pass and tokens one by one give the logits of the whole sequence at once.

    Both sides round alike except for the order of sums and, in bf16, the roundings between the operators
    (2^-8 each, a dozen of them): 2^-4 of the largest logit in bf16, 2^-14 in fp32."""
    log("decode %s prompt %d" % (dtype, prompt))
    model = ex.Model(64, dtype=dtype)
    B, L = 4, 60
    tokens = torch.randint(0, ex.VOCAB, (B, L), generator=torch.Generator().manual_seed(7)).to(DEV)
    with torch.no_grad():
        whole = model(tokens).float()
    tol = (2.0 ** -4 if dtype == torch.bfloat16 else 2.0 ** -14) * whole.abs().max()
    dec = ex.Decoder(model, B)
    out = dec.prefill(tokens[:, :prompt]).float()
    assert (out - whole[:, :prompt]).abs().max() <= tol
    for t in range(prompt, L):
        assert (dec.step(tokens[:, t]).float() - whole[:, t]).abs().max() <= tol, t
    assert torch.all(dec.pos == L)


def test_training_lowers_the_loss():
    """Forty steps on the repeat task: below the loss of knowing nothing (log 32) by a clear margin at its start."""
    losses = ex.train(ex.Model(128), 40, log=log)
    assert np.isfinite(losses).all()
    assert np.mean(losses[-5:]) < np.mean(losses[:5]) - 0.5
