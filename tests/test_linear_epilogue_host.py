"""nvq_linear_epilogue has one set of rules, whichever path it takes (no GPU: refused before anything is launched)."""
import ctypes

import pytest

import phase_disaggregated_quantized_b200 as nvq
from phase_disaggregated_quantized_b200 import build_lib

FAKE = 0x7F0000000000          # 16-byte aligned, never dereferenced: validation fails first
FAR = FAKE + (1 << 40)


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return nvq.lib()


@pytest.mark.parametrize("crossover", [0, 1 << 20])
@pytest.mark.parametrize("x, y, ldy", [
    (FAKE, FAKE, 0),                                          # the same matrix
    (FAKE, FAKE + 2 * 256 * 63, 0),                           # y begins in x's last row
    (FAKE + 2 * 256 * 63, FAKE, 0),                           # x begins in y's last row
    (FAKE + 2 * 512 * 63 + 2 * 248, FAKE, 512),               # in the last row of a y with a stride
])
def test_x_may_not_overlap_y_on_either_path(L, crossover, x, y, ldy):
    M, N, K = 64, 256, 256
    e = ctypes.byref(nvq.Epilogue(None, None, 0, ldy, 0))
    vp = ctypes.c_void_p
    got = L.nvq_linear_epilogue(vp(x), M, N, K, vp(FAR), vp(FAR), vp(FAR), vp(FAR), vp(FAR), crossover, vp(y), e, vp(FAR), 1 << 40, None)
    assert got == 1 and b"x overlaps y" in L.nvq_last_error_detail()
