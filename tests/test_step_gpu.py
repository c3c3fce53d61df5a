"""One token at a time on the GPU: scan_step, conv_step and conv_cache_fill."""
import math

import numpy as np
import pytest
import torch

import gated_convolution_sequence_amd as hc
import layer_ref as ref
import oracle
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


def rows(B, D, n, dtype, seed, fused=False):
    gen = torch.Generator().manual_seed(seed)
    big = torch.randn(B, n * D, generator=gen).to(dtype).to(DEV)
    ts = [big[:, i * D:(i + 1) * D] for i in range(n)]
    return ts if fused else [t.contiguous() for t in ts]


@pytest.mark.parametrize("B,S,D", [(1, 1, 1), (1, 1, 4096), (3, 5, 7), (2, 2, 72), (40, 64, 130), (257, 300, 64),
                                   (5, 9, 1001)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("gate", ["sigmoid", "log"])
@pytest.mark.parametrize("inplace", [True, False])
def test_scan_step(B, S, D, dtype, gate, inplace):
    log("scan_step %d %d %d %s %s" % (B, S, D, dtype, gate))
    q, k, v, g = rows(B, D, 4, dtype, B * D, fused=B % 2 == 1)
    if gate == "log":
        g.copy_(-g.abs())
    gen = torch.Generator().manual_seed(1)
    slots = torch.randperm(S, generator=gen)[:B].to(torch.int32)
    if B > 4:
        slots[1], slots[3] = -1, S  # two inactive entries
        g[2, 0] = -math.inf
    state = torch.randn(S, D, generator=gen).to(DEV)
    if B > 4:
        state[slots[2].item(), 0] = math.nan  # dropped by the closed gate
    before = state.clone()
    other = torch.full_like(state, 3.0)
    y = hc.scan_step(q, k, v, g, state, slots=slots.to(DEV), gate=gate, state_out=None if inplace else other)
    after = state if inplace else other
    if not inplace:
        assert torch.equal(torch.nan_to_num(state, 9.0), torch.nan_to_num(before, 9.0))
    live = [b for b in range(B) if 0 <= slots[b] < S]
    a, _ = ref.decay(to_np(g)[live], gate)
    old = to_np(before)[slots[live].numpy()]
    x = to_np(k)[live] * to_np(v)[live]
    kept = np.where(a == 0, 0.0, a * old)
    s = kept + x
    es = (np.minimum(np.abs(to_np(g)[live]), 1e30) + 10) * U * np.abs(kept) + 2 * U * (np.abs(kept) + np.abs(x))
    check(after[slots[live].long().to(DEV)], s, es, F32, "state")
    check(y[torch.tensor(live, device=DEV)], to_np(q)[live] * s, np.abs(to_np(q)[live]) * (es + U * np.abs(s)), dtype, "y")
    dead = [b for b in range(B) if b not in live]
    assert torch.all(y[dead] == 0)
    untouched = [i for i in range(S) if i not in slots.tolist()]
    assert torch.equal(after[untouched], (before if inplace else torch.full_like(before, 3.0))[untouched])


def test_scan_steps_follow_the_scan():
    """A prompt by scan_fwd and tokens by scan_step are the whole sequence by scan_fwd."""
    B, L, D, cut = 3, 90, 136, 77
    gen = torch.Generator().manual_seed(3)
    ts = [torch.randn(B, L, D, generator=gen).to(DEV) for _ in range(4)]
    f = ref.scan_fwd(*(to_np(t) for t in ts), "sigmoid")
    y, state, _ = hc.scan_fwd(*(t[:, :cut].contiguous() for t in ts))
    for t in range(cut, L):
        yt = hc.scan_step(*(x[:, t] for x in ts), state)
        check(yt, f["y"][:, t], f["ey"][:, t], F32, "row %d" % t)


def conv_ref(q, k, v, h, gs):
    a = [to_np(t) for t in (q, k, v, h)]
    return oracle.conv_fwd_ref(*a, gs), oracle.conv_fwd_ref(*(np.abs(x) for x in a), gs)


def conv_check(y, want, env, l_h, dtype, what):
    """x in the cache is rounded once (2^-8 in bf16); sums of l_h products in fp32."""
    op = 2.0 ** -8 * (1 + 2.0 ** -8) if dtype == BF16 else U
    check(y, want, (op + (l_h + 4) * U) * env, dtype, what)


@pytest.mark.parametrize("B,D,gs,l_h,R", [(1, 16, 16, 1, 1), (2, 64, 16, 7, 7), (3, 72, 8, 12, 16), (1, 7, 7, 5, 6),
                                          (2, 33, 1, 33, 40), (2, 256, 16, 128, 128), (5, 40, 2, 65, 130),
                                          (1, 4096, 16, 7, 8), (2, 24, 12, 3, 4)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_conv_steps_are_the_convolution(B, D, gs, l_h, R, dtype):
    """From an empty ring (its contents NaN), token by token past the ring's end, against the oracle."""
    log("conv_step %s %s" % ((B, D, gs, l_h, R), dtype))
    L = 2 * R + 3 if R < 60 else R + 9
    gen = torch.Generator().manual_seed(D + l_h)
    q, k, v = (torch.randn(B, L, D, generator=gen).to(dtype).to(DEV) for _ in range(3))
    h = (torch.randn(D // gs, l_h, generator=gen) / math.sqrt(l_h)).to(dtype).to(DEV)
    want, env = conv_ref(q, k, v, h, gs)
    S = B + 2
    slots = torch.randperm(S, generator=gen)[:B].to(torch.int32).to(DEV)
    cache = torch.full((S, R, D), float("nan"), dtype=dtype, device=DEV)
    pos = torch.zeros(B, dtype=torch.int64, device=DEV)
    for t in range(L):
        y = hc.conv_step(q[:, t], k[:, t], v[:, t], h, cache, pos, gs, slots=slots)
        conv_check(y, want[:, t], env[:, t], l_h, dtype, "row %d" % t)
        pos += 1
    x = (k.float() * v.float()).to(dtype)
    for t in range(L - R, L):
        assert torch.equal(cache[slots.long(), t % R], x[:, t])
    idle = [i for i in range(S) if i not in slots.tolist()]
    assert torch.isnan(cache[idle]).all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,fused", [(64, True), (72, False), (9, True)])
def test_prompts_of_any_length_then_steps(dtype, D, fused):
    """Ragged prompts (none, one row, longer than the ring) fill the rings; the next tokens continue them."""
    gs, l_h, R, L, more = 1, 20, 24, 100, 6
    lens = [0, 1, 19, 20, 24, 25, 60, 94]
    B = len(lens)
    gen = torch.Generator().manual_seed(D)
    big = torch.randn(B, L, 3 * D, generator=gen).to(dtype).to(DEV)
    q, k, v = (big[:, :, i * D:(i + 1) * D] for i in range(3))
    if not fused:
        q, k, v = (t.contiguous() for t in (q, k, v))
    h = (torch.randn(D, l_h, generator=gen) / math.sqrt(l_h)).to(dtype).to(DEV)
    want, env = conv_ref(q, k, v, h, gs)
    cache = torch.full((B + 1, R, D), 5.0, dtype=dtype, device=DEV)
    slots = torch.tensor([3, 1, 2, 0, 7, 5, 8, 4], dtype=torch.int32, device=DEV)
    pos = torch.tensor(lens, dtype=torch.int64, device=DEV)
    hc.conv_cache_fill(k, v, cache, lens=pos, slots=slots)
    assert torch.all(cache[6] == 5.0)
    x = (k.float() * v.float()).to(dtype)
    for b, n in enumerate(lens):
        ring = cache[slots[b].item()]
        for t in range(max(0, n - R), n):
            assert torch.equal(ring[t % R], x[b, t])
        for r in range(n, R):
            assert torch.all(ring[r] == 5.0)
    for i in range(more):
        idx = pos[:, None, None].expand(B, 1, D)
        y = hc.conv_step(*(t.gather(1, idx)[:, 0] for t in (q, k, v)), h, cache, pos, gs, slots=slots)
        w = np.stack([want[b, lens[b] + i] for b in range(B)])
        e = np.stack([env[b, lens[b] + i] for b in range(B)])
        conv_check(y, w, e, l_h, dtype, "step %d" % i)
        pos += 1


def test_conv_step_inactive_entries():
    B, D = 4, 64
    q, k, v = rows(B, D, 3, BF16, 5)
    h = torch.ones(4, 3, dtype=BF16, device=DEV)
    cache = torch.full((2, 4, D), 2.0, dtype=BF16, device=DEV)
    pos = torch.tensor([5, -1, 0, 7], dtype=torch.int64, device=DEV)
    slots = torch.tensor([-1, 0, 2, 1], dtype=torch.int32, device=DEV)
    y = hc.conv_step(q, k, v, h, cache, pos, 16, slots=slots)
    assert torch.all(y[:3] == 0) and not torch.all(y[3] == 0)
    assert torch.all(cache[0] == 2.0) and torch.all(cache[1, [0, 1, 2]] == 2.0)
    assert torch.equal(cache[1, 3], (k[3].float() * v[3].float()).to(BF16))


def test_a_long_way_in():
    """Positions past 32 bits; a pool of rings past 4 GiB."""
    R, D, S = 128, 4096, 4200  # 4.4 GB
    cache = torch.zeros((S, R, D), dtype=BF16, device=DEV)
    q, k, v = rows(1, D, 3, BF16, 6)
    h = torch.randn(D // 16, 100, device=DEV).to(BF16)
    slots = torch.tensor([S - 1], dtype=torch.int32, device=DEV)
    pos = torch.tensor([(1 << 33) + 5], dtype=torch.int64, device=DEV)
    cache[S - 1] = torch.randn(R, D, device=DEV).to(BF16)
    past = to_np(cache[S - 1])
    y = hc.conv_step(q, k, v, h, cache, pos, 16, slots=slots)
    x = np.stack([past[(5 - s) % R] for s in range(1, 100)])
    taps = to_np(h).repeat(16, axis=0)
    x0 = to_np(k)[0] * to_np(v)[0]
    want = to_np(q)[0] * (taps[:, 0] * x0 + (taps[:, 1:].T * x).sum(0))
    env = np.abs(to_np(q)[0]) * (np.abs(taps[:, 0] * x0) + np.abs(taps[:, 1:].T * x).sum(0))
    check(y[0], want, 104 * U * env, BF16, "y")
    assert torch.equal(cache[S - 1, 5], (k[0].float() * v[0].float()).to(BF16))


def test_steps_in_a_graph():
    """A decode step of both mixers captured once: the host only replays it."""
    B, D, l_h, R = 4, 128, 7, 8
    gen = torch.Generator().manual_seed(8)
    seq = torch.randn(6, B, 4 * D, generator=gen).to(BF16).to(DEV)
    h = torch.randn(D // 16, l_h, generator=gen).to(BF16).to(DEV)

    def fresh():
        return (torch.zeros(B, D, device=DEV), torch.zeros(B, R, D, dtype=BF16, device=DEV),
                torch.zeros(B, dtype=torch.int64, device=DEV))

    def step(row, state, cache, pos):
        q, k, v, g = (row[:, i * D:(i + 1) * D] for i in range(4))
        y = hc.scan_step(q, k, v, g, state), hc.conv_step(q, k, v, h, cache, pos, 16)
        pos += 1
        return y

    static, st = seq[0].clone(), fresh()
    step(static, *st)
    for t in st:
        t.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(static, *st)
    for t in st:
        t.zero_()
    eager = fresh()
    for r in range(6):
        static.copy_(seq[r])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step(seq[r], *eager)):
            assert torch.equal(a, b), "replay %d" % r


def test_refusals():
    t = torch.zeros(2, 16, dtype=BF16, device=DEV)
    state = torch.zeros(2, 16, device=DEV)
    cache = torch.zeros(2, 8, 16, dtype=BF16, device=DEV)
    pos = torch.zeros(2, dtype=torch.int64, device=DEV)
    h = torch.zeros(1, 7, dtype=BF16, device=DEV)
    with pytest.raises(ValueError):
        hc.scan_step(t, t, t, t, state.to(BF16))
    with pytest.raises(ValueError):
        hc.scan_step(t, t, t, t, state, slots=torch.zeros(2, dtype=torch.int64, device=DEV))
    with pytest.raises(hc.LayerError) as e:  # fewer states than sequences
        hc.scan_step(t, t, t, t, state[:1])
    assert e.value.status == -2
    with pytest.raises(hc.LayerError) as e:  # a ring shorter than the filter
        hc.conv_step(t, t, t, h, cache[:, :6].contiguous(), pos, 16)
    assert e.value.status == -2
    with pytest.raises(hc.LayerError) as e:
        hc.conv_step(t, t, t, torch.zeros(1, 129, dtype=BF16, device=DEV),
                     torch.zeros(2, 200, 16, dtype=BF16, device=DEV), pos, 16)
    assert e.value.status == -4
    with pytest.raises(ValueError):
        hc.conv_step(t, t, t, h, cache, pos.to(torch.int32), 16)
    with pytest.raises(ValueError):
        hc.conv_step(t, t, t, h, cache, pos, 5)
    with pytest.raises(ValueError):
        hc.conv_cache_fill(t[None], t[None], cache.float())
