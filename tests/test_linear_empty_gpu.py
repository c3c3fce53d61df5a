"""linear_bwd and LinearAct with sizes of 0 and only some gradients wanted."""
import pytest
import torch

import gated_convolution_sequence_amd as hc
from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(0, 6, 8), (4, 0, 8), (4, 6, 0), (0, 0, 8), (0, 6, 0), (4, 0, 0), (0, 0, 0)])
@pytest.mark.parametrize("need", [(a, b, c) for a in (0, 1) for b in (0, 1) for c in (0, 1)], ids=str)
@pytest.mark.parametrize("act", ["none", "silu"])
def test_any_gradients_of_any_empty_size(M, N, K, need, act):
    e = lambda *s: torch.randn(*s, device=DEV).to(torch.bfloat16)  # noqa: E731
    x, w, dy, z = e(M, K), e(N, K), e(M, N), e(M, N)
    got = hc.linear_bwd(x, w, dy, preact=z if act != "none" else None, act=act, need_dx=bool(need[0]),
                        need_dw=bool(need[1]), need_db=bool(need[2]))
    for n, g, shape in zip(need, got, ((M, K), (N, K), (N,))):
        assert (g is not None) == bool(n)
        if n:
            assert g.shape == shape
    if need[0] and M and K:
        assert torch.all(got[0] == 0)
    if need[1] and N and K:
        assert torch.all(got[1] == 0)
    if need[2] and M == 0:
        assert torch.all(got[2] == 0)


def test_an_empty_batch_with_frozen_weights():
    x = torch.empty(0, 8, dtype=torch.bfloat16, device=DEV, requires_grad=True)
    w = torch.randn(6, 8, device=DEV).to(torch.bfloat16)
    hc.LinearAct.apply(x, w, None, None, "silu").sum().backward()
    assert x.grad.shape == (0, 8)
