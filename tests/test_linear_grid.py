"""Row tiles of kda_linear's launches: the grid's y ends at 65535, whatever M and K."""
import ctypes

import pytest

from gated_delta_rule_46_gb300 import kda


@pytest.mark.parametrize("out", [kda.KDA_BF16, kda.KDA_F32])
@pytest.mark.parametrize("K", [1, 64, 512, 513, 2048, 2056, 4096, 4104, 65536, (1 << 31) - 1])
@pytest.mark.parametrize("M", [1, 64, 257, 1 << 22, 4194241, 1 << 23, 8388609, (1 << 31) - 1])
def test_row_tiles_fit_the_grid(M, K, out):
    f = kda.lib().kda_testing_linear_row_tiles
    f.restype, f.argtypes = ctypes.c_int64, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
    assert 1 <= f(M, K, out) <= 65535
