"""Every row's part in the readout's dw and db, by sums of whole numbers.

Bounds for sums of floats grow with the number of rows until a missing row is smaller
than they are.  Here logits and lse are 0, so that a row adds dloss x to each entry but
its target, whole numbers of a few units: partial sums are exact in fp32 in any order.
Rows cancel in random pairs but for a few, so that what comes out is small, exact in bf16
as well, and one row more or less changes it."""
import pytest
import torch

import gated_convolution_sequence_amd as hc

BF16, F32 = torch.bfloat16, torch.float32
SHAPES = [(8, 3, BF16), (8, 3, F32), (100, 4, F32), (264, 2, BF16), (1, 130, BF16), (72, 40, BF16), (77, 500, F32)]
ROWS = [5, 17, 200, 4097, 8191, 8192, 8193, 16384, 70001]


def rows_of(M, K, V, masked, alike, seed=0):
    """x, target, dloss (CPU, 32 bits).  alike: dloss is 1 everywhere and pairs cancel by x, in dw only."""
    gen = torch.Generator().manual_seed(seed)
    target = torch.randint(0, V, (M,), generator=gen)
    x = torch.randint(1, 4, (M, K), generator=gen) * (1 - 2 * torch.randint(0, 2, (M, K), generator=gen))
    on = torch.nonzero(torch.rand(M, generator=gen) >= masked)[:, 0]
    order = on[torch.randperm(len(on), generator=gen)]
    first, second = order[5::2], order[6::2]
    first = first[:len(second)]
    dloss = torch.ones(M)
    target[second] = target[first]
    if alike:
        x[second] = -x[first]
    else:
        x[second] = x[first]
        dloss[order[:5]] = torch.tensor([1.0, -1.0, 1.0, 1.0, -1.0])[:min(5, len(order))]
        dloss[second] = -dloss[first]
    off = torch.ones(M, dtype=torch.bool)
    off[on] = False
    target[off] = torch.where(torch.arange(M) % 2 == 0, -100, V)[off]
    return x.float(), target, dloss, on


def sums_of(x, target, dloss, on, V):
    """dw [V, K] and db [V] in 64 bits, of the rows `on`."""
    d = dloss[on].double()
    e = (1 - torch.nn.functional.one_hot(target[on], V).double()) * d[:, None]
    return e.t() @ x[on].double(), e.sum(0)


@pytest.mark.parametrize("K,V,dtype", SHAPES)
@pytest.mark.parametrize("M", ROWS)
def test_a_row_more_or_less_shows(M, K, V, dtype):
    """Of the sums themselves, on the CPU: exact in the output's type, and what some rows add to them is not 0."""
    for masked in (0.0, 0.5):
        for alike in (False, True):
            x, target, dloss, on = rows_of(M, K, V, masked, alike)
            dw, db = sums_of(x, target, dloss, on, V)
            assert torch.equal(dw.to(dtype).double(), dw) and int(x.abs().sum(0).max()) < 1 << 24
            assert alike or torch.equal(db.to(dtype).double(), db)
            for n in (1, 17, 49, 200, 1000):  # the last rows
                assert n >= len(on) or sums_of(x, target, dloss, on[-n:], V)[0].any(), n
            for i in range(0, len(on), max(1, len(on) // 16)):  # one row
                less = sums_of(x, target, dloss, on[i:i + 1], V)
                assert less[0].any() and less[1].any(), i


@pytest.mark.gpu
@pytest.mark.parametrize("K,V,dtype", SHAPES)
@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("masked", [0.0, 0.5, 0.99])
@pytest.mark.parametrize("alike", [False, True])
def test_every_row_is_in_the_sums(M, K, V, dtype, masked, alike):
    """dw and db to the bit, with rows without a target holding NaN; both products together, and each alone."""
    dev = torch.device("cuda:0")
    x, target, dloss, on = rows_of(M, K, V, masked, alike)
    dw, db = sums_of(x, target, dloss, on, V)
    off = torch.ones(M, dtype=torch.bool)
    off[on] = False
    x[off], dloss[off] = float("nan"), float("nan")
    args = (x.to(dev, dtype), torch.zeros(V, K, dtype=dtype, device=dev), target.to(dev), torch.zeros(M, device=dev),
            dloss.to(dev))
    bias = torch.zeros(V, dtype=dtype, device=dev)
    for need_dx in (True, False):
        dx, got_w, got_b = hc.xent_bwd(*args, bias=bias, need_dx=need_dx)
        assert torch.equal(got_w.cpu().double(), dw)  # exact in either type
        assert torch.equal(got_b.cpu(), db.to(dtype))
        assert dx is None or not dx.any()
    assert torch.equal(hc.xent_bwd(*args, need_dx=False)[1], got_w)
