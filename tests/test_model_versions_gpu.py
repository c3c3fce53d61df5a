"""What the model operators write into given tensors is seen by autograd: a graph that saved one refuses its backward."""
import math

import pytest
import torch

import gated_convolution_sequence_amd as hc
from gpu_util import DEV

pytestmark = pytest.mark.gpu
F32, F8 = torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    hc.model_lib()
    yield
    torch.cuda.synchronize()


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


def lists(sizes, bits=32):
    t = dict(params=[randn(*n, seed=1) for n in sizes], grads=[randn(*n, seed=2) for n in sizes],
             masters=[randn(*n, seed=1) for n in sizes])
    for name in ("exp_avgs", "exp_avg_sqs"):
        if bits == 32:
            t[name] = [torch.zeros(*n, device=DEV) for n in sizes]
        else:
            t[name] = [torch.zeros(*n, dtype=torch.uint8, device=DEV).view(F8) for n in sizes]
            t[name[:-1] + "_scales"] = [torch.zeros(-(-math.prod(n) // 256), device=DEV) for n in sizes]
    return t


@pytest.mark.parametrize("which", ["x", "w", "bias"])
def test_a_graph_kept_across_a_step_refuses_its_backward(which):
    """The lse and the statistics that a graph saved belong to the weights before the step."""
    leaves = dict(x=randn(40, 16), w=randn(60, 16, seed=3), bias=randn(60, seed=4))
    leaves = {k: v.requires_grad_(True) for k, v in leaves.items()}
    target = torch.arange(40, device=DEV)
    y = hc.Norm.apply(leaves["x"], None, None, "rms", 1e-5)
    loss = hc.LinearXent.apply(y, leaves["w"], target, leaves["bias"]).sum()
    first = torch.autograd.grad(loss, list(leaves.values()), retain_graph=True)
    p = leaves[which]
    with torch.no_grad():
        hc.adamw_step([p], [torch.ones_like(p)], [torch.zeros_like(p)], [torch.zeros_like(p)], step=1, lr=1e-2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(loss, list(leaves.values()))
    # a graph of the new weights is as good as any
    y = hc.Norm.apply(leaves["x"], None, None, "rms", 1e-5)
    loss = hc.LinearXent.apply(y, leaves["w"], target, leaves["bias"]).sum()
    assert not torch.equal(torch.autograd.grad(loss, list(leaves.values()))[1], first[1])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("masters", [True, False])
def test_a_step_raises_the_versions_of_what_it_writes(bits, masters):
    t = lists([(30, 9), (0,), (700,)], bits)
    if not masters:
        del t["masters"]
    before = {k: [x._version for x in ts] for k, ts in t.items()}
    hc.adamw_step(**t, step=1, lr=1e-2)
    for k, ts in t.items():
        for x, old in zip(ts, before[k]):
            assert (x._version == old) if k == "grads" else (x._version > old), k
    # a call that is refused writes nothing
    before = {k: [x._version for x in ts] for k, ts in t.items()}
    with pytest.raises(hc.ModelError):
        hc.adamw_step(**t, step=0, lr=1e-2)
    assert before == {k: [x._version for x in ts] for k, ts in t.items()}


def test_a_tensor_whose_rows_are_the_list():
    """Sequences of any kind: the rows of one tensor each, whose versions are the tensor's."""
    t = {k: randn(3, 50, seed=i) for i, k in enumerate(("params", "grads", "masters", "exp_avgs"))}
    t["exp_avg_sqs"] = t["exp_avgs"].square()
    want = {k: [x.clone() for x in v] for k, v in t.items()}
    hc.adamw_step(**want, step=3, lr=1e-2)
    before = {k: v._version for k, v in t.items()}
    hc.adamw_step(**t, step=3, lr=1e-2)
    for k, v in t.items():
        assert torch.equal(v, torch.stack(want[k])) and (v._version > before[k]) == (k != "grads"), k


def test_steps_of_inference_tensors():
    """They have no version; a step in inference mode, and outside of it, takes them as they are."""
    with torch.inference_mode():
        t = lists([(50,)])
        hc.adamw_step(**t, step=1, lr=1e-2)
    hc.adamw_step(**t, step=2, lr=1e-2)


def test_outputs_that_are_given():
    x, w = randn(20, 24), randn(24, seed=1)
    y, mean, rstd = hc.norm_fwd(x, w, save_stats=True)
    out, keep = torch.empty_like(x), torch.ones_like(x, requires_grad=True)
    for call in (lambda: hc.norm_fwd(x, w, out=out),
                 lambda: hc.norm_bwd(x, w, y, mean, rstd, dx=out),
                 lambda: hc.xent_bwd(x, randn(30, 24), torch.arange(20, device=DEV), rstd, rstd, dx=out)):
        kept = (keep * out.copy_(x)).sum()
        call()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            kept.backward()
    version = out._version
    hc.norm_bwd(x, w, y, mean, rstd, need_dx=False, dx=out)  # not written
    assert out._version == version
