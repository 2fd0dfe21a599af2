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


def up(a, b):
    return -(-a // b) * b


@pytest.mark.parametrize("k", [0, 8, 1024])
@pytest.mark.parametrize("T,V,D", [(1, 1, 8), (7, 1000, 72), (32, 131072, 4096), (33, 131072, 4096), (128, 4200000, 1000), (129, 50021, 2056), (3000, 50021, 2056),
                                   (16384, 131072, 4096), (131072, 131072, 4096), (1 << 20, 1000, 64), (1 << 24, 1000, 64), (1 << 24, 1 << 24, 8),
                                   (5000, 1 << 20, 64), (5000, (1 << 20) + 8, 64), (5000, 1 << 24, 64)])
def test_workspace_is_what_the_header_says(gemm_lib, T, V, D, k):
    size, w = gemm_lib.lib().gemm_relu_loss_workspace, up(D, 64)
    stats = 12 * up(V, 64) // 64
    most = max(2048, min(16384, (384 << 20) // stats // 256 * 256))
    R = T if T <= most else up(-(-T // -(-T // most)), 256)
    rest = 128 * R + (24 << 10)
    need = size(T, V, D, k, 0)
    told = stats * R + (2 * R * w if T > 128 else 0) + 8 * R * k
    assert told <= need <= told + rest + 32 * stats, (need, told)
    rows = 2 * up(T, 8) if T <= 32 else T
    P = max(256, (512 << 20) // (2 * rows) // 256 * 256)
    P = up(-(-V // -(-V // P)), 256)
    need = size(T, V, D, k, 1)
    told = 2 * rows * P + 2 * rows * w + 8 * T * k
    share = 4 * rows * D
    assert told + share <= need <= told + 64 * share + 128 * T + (24 << 10), (need, told, share)
    assert (need - told) // share <= 64 or T < 32


def test_caps_of_the_workspace(gemm_lib):
    """The statistics' 384 MiB hold up to 2^20 words, G's 512 MiB up to 2^20 rows; 2^24 of either take 2048 rows' and 256 words'."""
    size = gemm_lib.lib().gemm_relu_loss_workspace
    assert size(1 << 24, 1 << 20, 8, 0, 0) < (384 << 20) + 16384 * (2 * 64 + 128) + (1 << 20)
    assert 6.4e9 < size(1 << 24, 1 << 24, 8, 0, 0) < 6.6e9
    assert size(1 << 20, 1 << 20, 8, 0, 1) < (512 << 20) + (1 << 20) * (64 * 4 * 8 + 2 * 64 + 128) + (1 << 20)
    assert 8.5e9 < size(1 << 24, 8, 8, 0, 1)
