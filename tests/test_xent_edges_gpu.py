"""Edges of the readout cross entropy: upstream gradients that are not finite."""
import math

import pytest
import torch

import gated_convolution_sequence_amd as hc
from gpu_util import DEV, log
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
