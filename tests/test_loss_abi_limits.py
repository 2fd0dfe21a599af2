"""The losses' entry points without a GPU: limits of their arguments."""
import ctypes

import pytest

import test_loss_abi as abi


@pytest.mark.parametrize("call", abi.TEACHER, ids=lambda f: f.__name__)
def test_temperatures(gemm_lib, call):
    """log2(e) / temperature has to be finite: 3e-39 and 4.2e-39 have a finite inverse, but not that."""
    L = gemm_lib.lib()
    for tau in (3e-39, 4.2e-39, 2e-45, 0.0, -2.0, float("inf"), float("nan")):
        assert call(L, tau=tau) == 1, tau
    for tau in (ctypes.c_float(1.2e-38).value, 1.0, 3e38):  # (refused for the workspace that is not there, behind this check)
        assert call(L, tau=tau, kind=3) == 1 and call(L, tau=tau, ws=abi.GOOD + 16) == 2, tau
