"""The model operators at sizes whose launches pass 2^32 work-items."""
import pytest
import torch

import gated_convolution_sequence_amd as hc
import model_ref as ref
from gpu_util import DEV, log
from model_ref import check

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    hc.model_lib()
    torch.cuda.empty_cache()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def test_logits_past_2_to_the_36():
    """2^36 fp32 logits and some are 2^24 tiles of 256 threads: rows of one period all come out alike, and right."""
    period, n, K, V = 1024, 1030, 4, (1 << 16) + 65
    log("readout of %d rows, %d entries" % (period * n, V))
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(period, K, generator=gen, device=DEV)
    w = torch.randn(V, K, generator=gen, device=DEV)
    target = torch.randint(-5000, V, (period,), generator=gen, device=DEV)
    loss, lse = hc.xent_fwd(x.repeat(n, 1), w, target.repeat(n))
    want = ref.xent_fwd(x, w, target, None)
    for got, r, what in ((loss, want[0], "loss"), (lse, want[1], "lse")):
        check(got[:period], *r, what)
        assert bool((got.view(n, period) == got[:period]).all()), what


def test_rows_past_2_to_the_29():
    """2^29 rows and some of one channel and two entries; dw and db are sums of whole numbers, in which each row shows.

    With logits and lse of 0 a row adds dloss x to the entry that is not its target.  Neighbours cancel but for
    their x, so that no partial sum passes what fp32 holds exactly."""
    period, n, V = 4096, (1 << 17) + 3, 2
    M = period * n
    log("readout of %d rows" % M)
    gen = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(period, 1, generator=gen, device=DEV).to(BF16)
    w = torch.tensor([[0.5], [-1.25]], device=DEV).to(BF16)
    target = torch.randint(-1, V, (period,), generator=gen, device=DEV)
    many, goal = x.repeat(n, 1), target.repeat(n)
    loss, lse = hc.xent_fwd(many, w, goal)
    want = ref.xent_fwd(x, w, target, None)
    for got, r, what in ((loss, want[0], "loss"), (lse, want[1], "lse")):
        check(got[:period], *r, what)
        assert bool((got.view(n, period) == got[:period]).all()), what
    dloss = torch.rand(period, generator=gen, device=DEV)
    dx, _, _ = hc.xent_bwd(many, w, goal, lse, dloss.repeat(n), need_dw=False)
    r = ref.xent_bwd(x, w, target, lse[:period], dloss, None, True)[0]
    check(dx[:period], *r, "dx")
    assert bool((dx.view(n, period) == dx[:period, 0]).all())
    del loss, dx, lse
    # the sums: dloss alternates, x = 1 but for the last row and one in the middle
    many.fill_(1.0), w.zero_()
    for row in (M - 1, (M // 2) | 1):
        goal[row] = goal[row - 1] = 0
        many[row] = 3.0
    goal[:] = goal.view(-1, 2)[:, :1].expand(-1, 2).reshape(-1)  # a pair has one target
    dloss = torch.tensor([1.0, -1.0], device=DEV).repeat(M // 2)
    _, dw, db = hc.xent_bwd(many, w, goal, torch.zeros(M, device=DEV), dloss, bias=torch.zeros(V, dtype=BF16, device=DEV),
                            need_dx=False)
    # each of the two rows adds -(3 - 1) to entry 1
    assert dw.flatten().tolist() == [0.0, -4.0] and not db.any()
