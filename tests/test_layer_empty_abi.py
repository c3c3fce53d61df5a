"""Outputs of no elements may be NULL, alone too (C ABI, without a GPU; the calls launch nothing)."""
import pytest

from test_layer_abi import built_library, linear_bwd, linear_fwd, scan_bwd, scan_fwd  # noqa: F401

NONE = dict(dx=None, dw=None, db=None)


@pytest.mark.parametrize("act", [0, 3])
@pytest.mark.parametrize("kw", [dict(M=0), dict(N=0, lddy=0), dict(K=0, ldx=0, lddx=0), dict(M=0, K=0, ldx=0, lddx=0),
                                dict(M=0, N=0, lddy=0)], ids=str)
def test_linear_bwd_with_only_empty_outputs(kw, act):
    assert linear_bwd(act=act, **NONE, **kw) == 0


def test_scan_with_only_empty_outputs():
    assert scan_fwd(L=0, y=None, last=None, states=None) == 0
    assert scan_bwd(L=0, dq=None, dk=None, dv=None, dg=None, ds0=None) == 0


def test_no_output_of_a_call_with_elements_is_refused():
    assert linear_bwd(**NONE) == -1 and linear_bwd(act=0, M=1, N=1, K=1, **NONE) == -1
    assert scan_fwd(L=1, y=None, last=None, states=None) == -1
    assert scan_bwd(L=1, dq=None, dk=None, dv=None, dg=None, ds0=None) == -1
    assert linear_fwd(y=None) == -1
