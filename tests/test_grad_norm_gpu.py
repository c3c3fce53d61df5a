"""The clipping scale under a bound that no norm reaches."""
import math

import pytest
import torch

import gated_convolution_sequence_amd as hc
from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_an_infinite_bound_scales_nothing_and_still_skips_what_is_not_finite(dtype):
    """min(1, inf / norm) is 1: a caller that does not clip, and wants steps of bad gradients skipped, says so with inf."""
    g = [torch.full((n,), 3.0, dtype=dtype, device=DEV) for n in (4, 0, 12)]
    norm, scale = hc.grad_norm(g, max_norm=math.inf)
    assert float(norm) == 12.0 and float(scale) == 1.0
    norm, scale = hc.grad_norm([torch.zeros(5, dtype=dtype, device=DEV)], max_norm=math.inf)
    assert float(norm) == 0.0 and float(scale) == 1.0
    for bad in (math.nan, math.inf, -math.inf):
        g[2][7] = bad
        norm, scale = hc.grad_norm(g, max_norm=math.inf)
        assert not math.isfinite(float(norm)) and math.isnan(float(scale))
