"""The model operators at sizes whose launches pass 2^32 work-items."""
import pytest
import torch

import gated_convolution_sequence_amd as hc
import model_ref as ref
from gpu_util import DEV, log
from model_ref import check

pytestmark = pytest.mark.gpu
BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


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


def states(n):
    """A parameter of n elements with moments in 8 bits."""
    def zeros(n, dtype):
        return torch.zeros(n, dtype=torch.uint8, device=DEV).view(dtype) if dtype is F8 else torch.zeros(n, dtype=dtype, device=DEV)

    blocks = -(-n // hc.STATE_BLOCK)
    return dict(params=zeros(n, BF16), exp_avgs=zeros(n, F8), exp_avg_sqs=zeros(n, F8), exp_avg_scales=zeros(blocks, F32),
                exp_avg_sq_scales=zeros(blocks, F32))


def same(a, b):
    """Equality of codes, scales or parameters, 2^30 elements at a time."""
    a, b = (x.view(torch.uint8) if x.dtype is F8 else x for x in (a, b))
    return all(bool((p == q).all()) for p, q in zip(a.split(1 << 30), b.split(1 << 30)))


def test_a_step_of_more_than_2_to_the_24_workgroups():
    """17 tensors of 2^31 elements and some with moments in 8 bits (2^24 workgroups hold 2^35; 142 GB): a step gives each
    what a call gives it that has only this tensor, at the same place in the list."""
    n, count = (1 << 31) + 77, 17
    log("adamw of %d x %d elements" % (count, n))
    gen = torch.Generator(device=DEV).manual_seed(3)
    grad = torch.empty(n, dtype=BF16, device=DEV)  # of all of them: it is only read
    for piece in grad.split(1 << 28):
        piece.normal_(generator=gen)
    kw = dict(step=1, lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1, seed=11)
    all_of = [states(n) for _ in range(count)]
    hc.adamw_step(grads=[grad] * count, **{k: [s[k] for s in all_of] for k in all_of[0]}, **kw)
    empty = states(0)
    for i in range(count):
        if i not in (0, 7, count - 1):
            assert same(all_of[i]["params"], all_of[0]["params"])
            continue
        alone = states(n)
        lists = {k: [empty[k]] * i + [alone[k]] for k in alone}
        hc.adamw_step(grads=[grad[:0]] * i + [grad], **lists, **kw)
        for k in alone:
            assert same(all_of[i][k], alone[k]), (i, k)
        assert bool(alone["params"][-77:].any()) and bool(alone["exp_avgs"][-77:].float().any())


def test_the_norm_of_more_than_2_to_the_24_workgroups():
    """2^34 gradients 49 times over, in two launches, the first of 1.5 x 2^24 workgroups: squares of 2^-20 add up exactly."""
    log("norm of 49 x 2^34 gradients")
    grad = torch.full((1 << 34,), 2.0 ** -10, dtype=BF16, device=DEV)
    norm, scale = hc.grad_norm([grad] * 49, max_norm=7.0)
    assert float(norm) == 7 * 2.0 ** 7 and float(scale) == 2.0 ** -7


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_a_row_past_2_to_the_28(dtype):
    """One row of 2^28 channels and some: dw = dy u and db = dy, with nothing to add up."""
    D = (1 << 28) + 4097
    log("norm backward of %d channels %s" % (D, dtype))
    gen = torch.Generator(device=DEV).manual_seed(4)
    x, dy = (torch.empty(1, D, dtype=dtype, device=DEV).normal_(generator=gen) for _ in range(2))
    w = torch.ones(D, dtype=dtype, device=DEV)
    mean, rstd = (torch.full((1,), v, device=DEV) for v in (0.25, 2.0))
    _, dw, db = hc.norm_bwd(x, w, dy, mean, rstd)
    assert torch.equal(db, dy[0])
    # u = (x - mean) rstd, a sum with one rounding and a product by a power of two; dy u one more
    want = (x[0].double() - 0.25) * 2 * dy[0].double()
    check(dw, want, 2 * ref.U * want.abs(), "dw")
