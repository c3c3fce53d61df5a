"""Calls of the model operators beside each other, from threads with a stream each: a call that raises fails the test."""
import threading
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import gated_convolution_sequence_amd as hc
from gpu_util import DEV

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
ROUNDS = 20


def jobs_of():
    """Each entry point's call on a given stream, with all that it writes."""
    gen = torch.Generator(device=DEV).manual_seed(5)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=DEV).to(BF16)

    x, w, b, dy = randn(3000, 512), randn(512), randn(512), randn(3000, 512)
    _, mean, rstd = hc.norm_fwd(x, w, b, save_stats=True)
    readout = randn(2000, 512) * 0.05
    target = torch.randint(-500, 2000, (3000,), generator=gen, device=DEV)
    _, lse = hc.xent_fwd(x, readout, target)
    dloss = torch.rand(3000, generator=gen, device=DEV)
    grads = [randn(n) for n in (7, 40000, 333)]

    def adam(bits, stream):
        p = [g.clone() for g in grads]
        kw, held = {}, torch.float32
        if bits == 8:
            kw = {k: [torch.zeros(-(-g.numel() // 256), device=DEV) for g in grads]
                  for k in ("exp_avg_scales", "exp_avg_sq_scales")}
            held = torch.uint8
        m, v = ([torch.zeros(g.shape, dtype=held, device=DEV) for g in grads] for _ in range(2))
        if bits == 8:
            m, v = ([t.view(torch.float8_e4m3fn) for t in ts] for ts in (m, v))
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        norm, scale = hc.grad_norm(grads, max_norm=1.0, stream=stream)
        hc.adamw_step(p, grads, m, v, step=2, lr=1e-2, grad_scale=scale, stream=stream, **kw)
        return (norm, scale, *p, *(t.view(torch.uint8) if bits == 8 else t for t in m + v), *(t for k in kw.values() for t in k))

    return [lambda s: hc.norm_fwd(x, w, b, save_stats=True, stream=s),
            lambda s: hc.norm_bwd(x, w, dy, mean, rstd, stream=s),
            lambda s: hc.xent_fwd(x, readout, target, stream=s), lambda s: hc.xent_fwd(x[:9], readout, target[:9], stream=s),
            lambda s: hc.xent_bwd(x, readout, target, lse, dloss, stream=s),
            lambda s: hc.xent_bwd(x[:9], readout, target[:9], lse[:9], dloss[:9], stream=s),
            lambda s: adam(32, s), lambda s: adam(8, s)]


def same(a, b):
    return len(a) == len(b) and all((p is None) == (q is None) and (p is None or torch.equal(p, q)) for p, q in zip(a, b))


def run_beside(jobs, alone):
    """How many rounds of each job gave the same as alone; what a thread raises is raised here."""
    together = threading.Barrier(len(jobs), timeout=60)

    def work(i):
        stream = torch.cuda.Stream()
        together.wait()
        done = 0
        for _ in range(ROUNDS):
            got = jobs[i](stream)
            stream.synchronize()
            done += same(got, alone[i])
        return done

    with ThreadPoolExecutor(len(jobs)) as pool:
        return [f.result(timeout=100) for f in [pool.submit(work, i) for i in range(len(jobs))]]


def test_calls_beside_each_other():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    jobs = jobs_of()
    alone = [job(None) for job in jobs]
    torch.cuda.synchronize()
    assert run_beside(jobs, alone) == [ROUNDS] * len(jobs)


def test_a_call_that_is_refused_beside_others_is_seen():
    """The harness's own check: one job's argument is refused, and no round of it counts."""
    jobs = jobs_of()[:2]
    alone = [job(None) for job in jobs]
    jobs[1] = lambda s: hc.norm_fwd(torch.zeros(3, 4, device=DEV), eps=-1.0, stream=s)
    torch.cuda.synchronize()
    with pytest.raises(hc.ModelError):
        run_beside(jobs, alone)
