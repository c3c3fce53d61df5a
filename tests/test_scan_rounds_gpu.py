"""The gated recurrence with more workgroups than the card holds at once, and with one tile counter.

Workgroups beyond the card's start only as others end, so carries are waited for across rounds; past
8192 workgroups all tiles come from one counter."""
import pytest
import torch

import gated_convolution_sequence_amd as hc
from gpu_util import log
from test_scan_gpu import check_bwd, check_fwd, inputs, states_of

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    hc.layer_lib()
    yield
    torch.cuda.synchronize()


def workgroups(B, L, D, dtype, rows):
    return -(-L // rows) * B * -(-D // (64 if dtype == F32 else 128))


# (shape, workgroups of the forward and of the backward at least): 512 and 768 fit the card's 256 units
@pytest.mark.parametrize("shape,dtype,gate,fwd,bwd", [
    ((8, 3000, 520), BF16, "sigmoid", 513, 769), ((3, 2900, 1000), F32, "log", 513, 769),
    ((136, 8190, 8), BF16, "log", 8193, 8193), ((130, 8200, 5), F32, "sigmoid", 8193, 8193),
])
def test_more_workgroups_than_fit(shape, dtype, gate, fwd, bwd):
    assert workgroups(*shape, dtype, 128) >= fwd and workgroups(*shape, dtype, 64) >= bwd
    log("scan rounds %s %s %s" % (shape, dtype, gate))
    ts = inputs(*shape, dtype, gate, sum(shape), resets=0.001)
    s0, ds_last = states_of(shape[0], shape[2], 1)
    _, _, states = check_fwd(ts, gate, s0, "fwd")
    got = check_bwd(ts, gate, s0, ds_last, states, "bwd")
    for a, b in zip(hc.scan_bwd(*ts, states, gate=gate, ds_last=ds_last), got):
        assert torch.equal(a, b)
