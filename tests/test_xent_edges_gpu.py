"""Edges of the readout cross entropy: upstream gradients that are not finite, tokens that are nearly certain,
fp32 logits of long rows."""
import math

import pytest
import torch

import gated_convolution_sequence_amd as hc
from gpu_util import DEV
from model_ref import U, check
from test_xent_gpu import inputs

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    hc.model_lib()
    yield
    torch.cuda.synchronize()


def with_target(t):
    V = t["w"].shape[0]
    return (t["target"] >= 0) & (t["target"] < V)


# ---- upstream gradients that are not finite --------------------------------------------

# dloss with x; with e (few entries for their length); rows that are packed for the logits
PATHS = [(64, 500), (72, 9), (77, 9)]


@pytest.mark.parametrize("M", [8, 200, 8192, 20000])
@pytest.mark.parametrize("K,V", PATHS)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("others", [NAN, 0.0, 0.3, -INF])
def test_nan_upstream_reaches_every_weight(M, K, V, dtype, others):
    """A dloss of NaN among rows of ``others``: all of dw and db are NaN, and dx where it belongs."""
    t = inputs(M, K, V, dtype, 31, masked=0.3)
    rows = torch.nonzero(with_target(t))[:, 0]
    _, lse = hc.xent_fwd(t["x"], t["w"], t["target"], bias=t["bias"])
    for at in {0, len(rows) // 2, len(rows) - 1}:
        d = torch.full_like(t["dloss"], others)
        d[rows[at]] = NAN
        for need_dx in (True, False):
            dx, dw, db = hc.xent_bwd(t["x"], t["w"], t["target"], lse, d, bias=t["bias"], need_dx=need_dx)
            assert torch.isnan(dw).all() and torch.isnan(db).all(), at
            if need_dx:
                assert torch.isnan(dx[rows[at]]).all()
                assert not math.isfinite(others) or torch.isfinite(dx[rows[rows != rows[at]]]).all()


@pytest.mark.parametrize("M", [8, 200, 20000])
@pytest.mark.parametrize("K,V", PATHS)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_upstream_of_rows_without_a_target_is_not_read(M, K, V, value):
    t = inputs(M, K, V, BF16, 32, masked=0.3)
    off = ~with_target(t)
    off[1], t["target"][1] = True, -1
    _, lse = hc.xent_fwd(t["x"], t["w"], t["target"], bias=t["bias"])
    for own in (0.0, 0.3):
        t["dloss"].fill_(own)
        want = hc.xent_bwd(t["x"], t["w"], t["target"], lse, t["dloss"], bias=t["bias"])
        t["dloss"][off] = value
        for a, b in zip(hc.xent_bwd(t["x"], t["w"], t["target"], lse, t["dloss"], bias=t["bias"]), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M", [8, 200, 20000])
@pytest.mark.parametrize("K,V", PATHS)
@pytest.mark.parametrize("value", [INF, -INF])
def test_infinite_upstream_leaves_no_weight_finite(M, K, V, value):
    t = inputs(M, K, V, BF16, 33, masked=0.3)
    rows = torch.nonzero(with_target(t))[:, 0]
    _, lse = hc.xent_fwd(t["x"], t["w"], t["target"], bias=t["bias"])
    for others in (0.0, 0.3, value):
        d = torch.full_like(t["dloss"], others)
        d[rows[len(rows) // 2]] = value
        dx, dw, db = hc.xent_bwd(t["x"], t["w"], t["target"], lse, d, bias=t["bias"])
        assert not torch.isfinite(dw).any() and not torch.isfinite(db).any()
        assert not torch.isfinite(dx[rows[len(rows) // 2]]).any()


# ---- tokens that are nearly certain ------------------------------------------------------

@pytest.mark.parametrize("M", [5, 60, 600])
@pytest.mark.parametrize("K", [2, 8])
@pytest.mark.parametrize("level", [0.0, 3968.0, -3968.0])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_the_loss_of_a_nearly_certain_token_keeps_its_digits(M, K, level, dtype):
    """Logits of level + 32 for the target and level + 13 to 20 for the others, exact in fp32: a loss of 0.0009.

    exp(z - the largest) sums to 1.0009: some 40 additions that round what is below 2 (lanes, waves, tiles), terms by
    their exponents' (20 + 2) U, and a logarithm.  lse, of thousands, has fewer digits than that; loss must not be
    formed from it."""
    V = 300
    w = torch.zeros(V, K, device=DEV)
    w[:, 0], w[:, 1] = level, 13.0 + torch.arange(V, device=DEV) % 8
    w[77, 1] = 32.0
    x = torch.zeros(M, K, device=DEV)
    x[:, :2] = 1.0
    target = torch.full((M,), 77, device=DEV)
    target[1::4] = 5
    loss, lse = hc.xent_fwd(x.to(dtype), w.to(dtype), target)
    d = w[:, 1].double()
    want = (torch.logsumexp(d - 32.0, 0) + 32.0 - d)[target]
    check(loss, want, 64 * U + 4 * U * want, "loss")
    check(lse, torch.logsumexp(level + d, 0).expand(M), 64 * U, "lse")


# ---- fp32 logits of long rows ------------------------------------------------------------

def chain_error(K):
    """The root mean square error of an fp32 logit over its own, for terms of random signs.

    A sum's n-th rounding is that of n terms' random walk: sqrt(n / N) of the last one's, at most 2^-24 / sqrt(3) in
    the mean square (a half unit, uniform).  Over a run of 256 terms, rounded once each at most, and the sums of
    K / 256 runs that comes to sqrt(256 / 2 + K / 256 / 2) of them; a quarter more for what 64 rows' mean may stray.
    (One chain over all K: sqrt(K / 2) of them, four to eleven times as much for the lengths below.)"""
    return 1.25 * 2.0 ** -24 / math.sqrt(3) * math.sqrt(128 + K / 512)


def rms(t):
    return float(t.double().square().mean().sqrt())


@pytest.mark.parametrize("M,V", [(64, 64), (200, 300)])
@pytest.mark.parametrize("K", [4096, 65536])
def test_fp32_logits_of_long_rows(M, V, K):
    gen = torch.Generator(device=DEV).manual_seed(41)
    x = torch.randn(M, K, generator=gen, device=DEV)
    w = torch.randn(V, K, generator=gen, device=DEV) * (25 * K ** -0.5)  # logits of some 25
    z = x.double() @ w.double().t()
    target = torch.arange(M, device=DEV) % V
    loss, lse = hc.xent_fwd(x, w, target)
    at = z.gather(1, target[:, None])[:, 0]
    err = rms(loss.double() - (torch.logsumexp(z, 1) - at))
    # of two logits, the largest and the target's, and the roundings of the loss and of its two parts
    most = chain_error(K) * math.hypot(rms(z.max(1).values), rms(at)) + 2 * U * rms(loss)
    assert err <= most
    # exp(z - lse) of single rows, as db shows them; lse of 0 leaves exp's (|z| + 2) U beside the logits' error
    zero, bias = torch.zeros(M, device=DEV), torch.zeros(V, device=DEV)
    rel = []
    for row in range(0, M, M // 16):
        only = torch.full_like(target, -1)
        only[row] = target[row]
        _, _, db = hc.xent_bwd(x, w, only, zero, zero + 1, bias=bias, need_dx=False, need_dw=False)
        keep = torch.arange(V, device=DEV) != target[row]
        keep &= z[row].abs() < 80
        rel.append((db.double() / z[row].exp() - 1)[keep])
    err = rms(torch.cat(rel))
    most = chain_error(K) * rms(z) + 27 * U
    assert err <= most
