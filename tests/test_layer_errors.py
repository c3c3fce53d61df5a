"""One exception type of the package catches the status of either library."""
import pytest

import gated_convolution_sequence_amd as hc
from test_layer_abi import built_library  # noqa: F401


def test_the_packages_error_catches_both_libraries():
    with pytest.raises(hc.HyenaError) as e:
        hc.scan_workspace_bytes(-1, 2, 3)
    assert isinstance(e.value, hc.LayerError) and e.value.status == -2
    assert str(e.value) == "hyena_scan_workspace: %s (-2)" % hc.layer_strerror(-2)
    with pytest.raises(hc.HyenaError) as e:
        hc.plan(-1, 2, 3, 1, 7)
    assert not isinstance(e.value, hc.LayerError)
