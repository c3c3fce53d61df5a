"""conv_step for large batches with filters of more than 32 taps: the kernels that keep 16 or 8 taps a lane.

They take over where ceil(D / 64) B (bf16; D / 32 in fp32) passes 1024: 16 taps where a lane's
channels share a filter, else 8 in two waves a sequence."""
import numpy as np
import pytest
import torch

import gated_convolution_sequence_amd as hc
from gpu_util import DEV, log
from layer_ref import U, check, to_np

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    hc.layer_lib()
    yield
    torch.cuda.synchronize()


def many(B, D, dtype):
    return -(-D // (32 if dtype == F32 else 64)) * B > 1024


# last items of a workgroup past D; D no whole number of vectors; groups narrower than a lane
@pytest.mark.parametrize("D,gs", [(520, 8), (576, 16), (1024, 16), (520, 2), (515, 1), (68, 4), (21, 1)])
@pytest.mark.parametrize("l_h,R", [(33, 33), (100, 128), (128, 131)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("strided", [False, True])
def test_large_batches(D, gs, l_h, R, dtype, strided):
    B = 1024 // -(-D // (32 if dtype == F32 else 64)) + 9
    S = B + 5
    assert many(B, D, dtype)
    log("conv_step batch %s %s" % ((B, D, gs, l_h, R), dtype))
    gen = torch.Generator().manual_seed(D + l_h)
    big = torch.randn(B, 3 * D + 1, generator=gen).to(dtype).to(DEV)
    q, k, v = (big[:, i * D + 1:(i + 1) * D + 1] for i in range(3))
    if not strided:
        q, k, v = (t.contiguous() for t in (q, k, v))
    h = (torch.randn(D // gs, l_h, generator=gen) / l_h ** 0.5).to(dtype).to(DEV)
    slots = torch.randperm(S, generator=gen)[:B].to(torch.int32)
    pos = torch.randint(l_h, 100000, (B,), generator=gen)
    pos[::8] = torch.randint(0, l_h, (len(pos[::8]),), generator=gen)  # younger than the filter
    pos[0], pos[1], pos[2], pos[3] = 0, 1, l_h - 1, (1 << 33) + 7
    slots[5], slots[B - 1], pos[6] = -1, S, -1  # inactive
    cache = torch.randn(S, R, D, generator=gen).to(dtype)
    # rows that no lag reaches hold NaN
    lag = torch.arange(1, l_h)
    live = [b for b in range(B) if 0 <= slots[b] < S and pos[b] >= 0]
    read = torch.zeros(S, R, dtype=torch.bool)
    for b in live:
        read[slots[b], (pos[b] - lag[lag <= pos[b]]) % R] = True
    cache[~read] = float("nan")
    before = cache.clone()
    cache, dev_pos, dev_slots = cache.to(DEV), pos.to(DEV), slots.to(DEV)
    y = hc.conv_step(q, k, v, h, cache, dev_pos, gs, slots=dev_slots)
    # tap by tap
    x = to_np(k) * to_np(v)
    taps = np.repeat(to_np(h), gs, axis=0)
    past, at = to_np(before), slots.long().clamp(0, S - 1).numpy()
    total, size = taps[:, 0] * x, np.abs(taps[:, 0] * x)
    for s in range(1, l_h):
        row = past[at, (pos.numpy() - s) % R]
        term = np.where((pos.numpy() >= s)[:, None], taps[:, s] * np.nan_to_num(row), 0.0)
        total, size = total + term, size + np.abs(term)
    want, env = to_np(q) * total, np.abs(to_np(q)) * size
    dead = [b for b in range(B) if b not in live]
    want[dead], env[dead] = 0.0, 0.0
    check(y, want, (l_h + 4) * U * env, dtype, "y")
    # each live ring has its new row, and nothing else moved
    expect = before.clone()
    xr = (k.float() * v.float()).to(dtype).cpu()
    for b in live:
        expect[slots[b], pos[b] % R] = xr[b]
    got = cache.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(expect))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(expect))


@pytest.mark.parametrize("D,gs", [(576, 16), (515, 1)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_a_large_batch_is_its_sequences_one_by_one(D, gs, dtype):
    """Each sequence alone takes another kernel, whose sums run in another order."""
    l_h, B = 120, 150
    assert many(B, D, dtype) and not many(3, D, dtype)
    gen = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(B, D, generator=gen).to(dtype).to(DEV) for _ in range(3))
    h = (torch.randn(D // gs, l_h, generator=gen) / l_h ** 0.5).to(dtype).to(DEV)
    cache = torch.randn(B, l_h, D, generator=gen).to(dtype).to(DEV)
    pos = torch.randint(0, 400, (B,), generator=gen).to(DEV)
    mine = cache.clone()
    whole = hc.conv_step(q, k, v, h, cache, pos, gs)
    size = to_np(hc.conv_step(q.abs(), k.abs(), v.abs(), h.abs(), mine.abs(), pos, gs).float())
    for b in (0, 1, 77, B - 1):
        ring = mine[b:b + 1].clone()
        one = hc.conv_step(q[b:b + 1], k[b:b + 1], v[b:b + 1], h, ring, pos[b:b + 1], gs)
        # sums of l_h terms, each off by (l_h + 4) u of the magnitudes (themselves rounded once)
        check(whole[b], to_np(one[0]), 2 * (l_h + 4) * U * 1.01 * size[b], dtype, "sequence %d" % b)
        assert torch.equal(cache[b], ring[0])
