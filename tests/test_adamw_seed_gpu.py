"""The random rounding of 8-bit moments where the caller gives no seed."""
import pytest
import torch

import gated_convolution_sequence_amd as hc
import model_ref as ref
from gpu_util import DEV
from test_adamw_gpu import F8, HYPER, copies, lists

pytestmark = pytest.mark.gpu
SIZES = [3000, 0, 257, 40000]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    hc.model_lib()
    yield
    torch.cuda.synchronize()


def after(t, **kw):
    t = copies(t)
    hc.adamw_step(**t, **HYPER, **kw)
    return t


def equal(a, b):
    return all(torch.equal(*(v.view(torch.uint8) if v.dtype == F8 else v for v in (x, y)))
               for k in a for x, y in zip(a[k], b[k]))


@pytest.mark.parametrize("step", [1, 2, 1000, (1 << 32) + 7])
def test_the_step_is_the_seed(step):
    """A number or a tensor, with the same bits as a seed of that number; another step has others."""
    t = lists(SIZES, torch.bfloat16, 1, True, bits=8)
    own = after(t, step=step)
    assert equal(own, after(t, step=step, seed=step))
    assert not equal(own, after(t, step=step, seed=step + 1))
    dev = torch.tensor([step], device=DEV)
    assert equal(own, after(t, step=dev)) and equal(own, after(t, step=dev, seed=step))


def test_moments_keep_moving_without_a_seed():
    """r = sqrt(v) from code 224 = 14 x 16 on, under a largest of 448 that stays: a step moves it by 0.3 % of a code.

    v goes from 1 towards 1.44 and reaches w = 1.44 - 0.44 beta2^steps in mean.  Rounding at random lifts E[c^2] over
    E[c]^2 by the variance, gap^2 p (1 - p) <= gap times r's move in each step, together at most gap (sqrt(w) - 1) = 0.004
    with gap = 1 / 14; and an element's v is spread by at most sqrt(gap 0.06) 2 < 0.14, the mean of 65280 of them by
    0.0006.  (The same bits in every step leave all but 0.3 % of the elements where they are: a mean of 1.00.)"""
    n, steps, beta2 = 1 << 16, 300, 0.999
    top = torch.arange(n, device=DEV) % 256 == 0  # of each block
    code = torch.where(top, 448.0, 224.0).to(F8)
    t = dict(params=[torch.zeros(n, device=DEV)], grads=[torch.where(top, 2.0, 1.2)], exp_avgs=[code.clone()],
             exp_avg_sqs=[code.clone()], exp_avg_scales=[torch.full((n // 256,), 1 / 224, device=DEV)],
             exp_avg_sq_scales=[torch.full((n // 256,), 1 / 224, device=DEV)])
    for step in range(1, steps + 1):
        hc.adamw_step(**t, step=step, lr=0.0, betas=(0.9, beta2))
    v = (ref.decode(t["exp_avg_sqs"][0], t["exp_avg_sq_scales"][0]) ** 2)[~top]
    assert abs(float(v.mean()) - (1.44 - 0.44 * beta2 ** steps)) < 0.004 + 5 * 0.0006


def test_a_captured_step_draws_anew_in_each_replay():
    t = lists(SIZES, torch.bfloat16, 2, True, bits=8)
    eager, step = copies(t), torch.ones(1, dtype=torch.int64, device=DEV)
    hc.adamw_step(**copies(t), step=step, **HYPER)  # loads what a first call loads
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hc.adamw_step(**t, step=step, **HYPER)
    for i in range(1, 5):
        step.fill_(i)
        graph.replay()
        hc.adamw_step(**eager, step=i, **HYPER)
        torch.cuda.synchronize()
        assert equal(t, eager), i
