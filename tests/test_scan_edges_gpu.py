"""The gated recurrence where rows past the end and values that are not finite meet its tiles.

Against the 64-bit walk of layer_ref, with its bounds."""
import math

import pytest
import torch

import gated_convolution_sequence_amd as hc
from gpu_util import DEV, log
from test_scan_gpu import check_bwd, check_fwd, inputs, states_of

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    hc.layer_lib()
    yield
    torch.cuda.synchronize()


# a whole number of tiles; 1, 2 and 3 rows of a lane's four; whole slices past the end; one row
@pytest.mark.parametrize("L", [1, 64, 65, 66, 67, 68, 100, 128, 190, 257])
@pytest.mark.parametrize("D", [64, 9])
@pytest.mark.parametrize("dtype,gate", [(BF16, "sigmoid"), (F32, "log")], ids=["bf16", "f32"])
def test_an_infinite_gradient_in_the_last_row(L, D, dtype, gate):
    """dy infinite in row L - 1: infinite gradients before it, NaN only where the formula has them."""
    log("scan infinite dy in row %d of D=%d %s" % (L - 1, D, dtype))
    ts = inputs(2, L, D, dtype, gate, 70 + L)
    s0, ds_last = states_of(2, D, 71)
    ts[4][0, L - 1, 3] = math.inf
    ts[4][1, L - 1, 0] = -math.inf
    ts[4][1, L - 1, D - 1] = math.inf
    ts[2][0, L - 1, 5] = math.inf  # v: only its own row's dk, and the last state
    _, _, states = check_fwd(ts, gate, s0, "fwd")
    dq, dk, dv, dg, ds0 = check_bwd(ts, gate, s0, ds_last, states, "bwd")
    assert torch.isinf(ds0[0, 3]) and torch.isinf(ds0[1, 0]) and not torch.isnan(ds0).any()
    assert not torch.isnan(dk).any()
