"""Host rules of the products with an epilogue: what is refused before anything is launched (no GPU)."""
import ctypes

import pytest
import torch

import phase_disaggregated_quantized_b200 as nvq
from phase_disaggregated_quantized_b200 import build_lib

FAKE = 0x7F0000000000          # 16-byte aligned, never dereferenced: validation fails first
FAR = FAKE + (1 << 40)
ODD = FAKE + 8


def _vp(v):
    return ctypes.c_void_p(v)


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return nvq.lib()


def _epi(bias=None, residual=None, ldr=0, ldy=0, act=0):
    return ctypes.byref(nvq.Epilogue(bias, residual, ldr, ldy, act))


def _calls(L, M, N, K, e, y=FAKE):
    """The same epilogue through the three products (packed and NVFP4 weights far from y)."""
    yield L.w4a16_gemm_epilogue(_vp(FAR), _vp(FAR), _vp(FAR), _vp(y), M, N, K, e, None)
    yield L.nvfp4_gemm_w4a4_epilogue(*([_vp(FAR)] * 6), _vp(y), M, N, K, e, None)
    ws = _vp(FAR)
    for crossover in (0, 1 << 20):
        yield L.nvq_linear_epilogue(_vp(FAR), M, N, K, _vp(FAR), _vp(FAR), _vp(FAR), _vp(FAR), _vp(FAR), crossover,
                                    _vp(y), e, ws, 1 << 40, None)


@pytest.mark.parametrize("e, want", [
    (dict(act=5), 1), (dict(act=-1), 1),
    (dict(ldy=248), 1), (dict(residual=FAR, ldr=128), 1), (dict(ldy=-256), 1),
    (dict(ldy=260), 3), (dict(residual=FAR, ldr=257), 3),
    (dict(ldy=1 << 31), 2),
    (dict(bias=FAR + 8), 3), (dict(residual=FAR + 8), 3),
    (dict(residual=FAKE + 16), 1),                              # one row group of y, shifted
    (dict(residual=FAKE + 512, ldr=256, ldy=256), 1),            # the next row of y
    (dict(residual=FAKE, ldr=512), 1),                           # y with another stride
    (dict(residual=FAKE + 2 * 128, ldr=512, ldy=512), 1),        # columns 128 .. 383 of y's buffer
    (dict(bias=FAKE + 512), 1),                                  # a row of y
])
def test_bad_epilogues_are_refused(L, e, want):
    for got in _calls(L, 64, 256, 512, _epi(**e)):
        assert got == want, nvq.lib().nvq_last_error_detail()


def test_bad_products_are_refused(L):
    e = _epi()
    g = L.w4a16_gemm_epilogue
    assert g(_vp(FAKE), _vp(FAR), _vp(FAR), _vp(FAR), 4, 48, 128, e, None) == 2       # N % 32
    assert g(_vp(FAKE), _vp(FAR), _vp(FAR), _vp(FAR), 4, 64, 100, e, None) == 2       # K % 128
    assert g(_vp(FAKE), _vp(FAR), _vp(FAR), _vp(FAR), -1, 64, 128, e, None) == 1
    assert g(_vp(FAKE), _vp(FAR), _vp(FAR), None, 4, 64, 128, e, None) == 1
    assert g(_vp(FAKE), _vp(FAR), _vp(FAR), _vp(FAR + 8), 4, 64, 128, e, None) == 3
    assert g(_vp(FAKE), _vp(FAR), _vp(FAR), _vp(FAKE + 256), 4, 64, 128, e, None) == 1   # y inside x
    assert g(_vp(FAKE), _vp(FAR), _vp(FAR), _vp(FAR), 0, 64, 128, e, None) == 0       # nothing to do
    f = L.nvfp4_gemm_w4a4_epilogue
    a = [_vp(FAR)] * 7
    assert f(*a, 128, 12, 512, e, None) == 2
    assert f(*a, 128, 512, 96, e, None) == 2
    assert f(*a, 1 << 24, 1 << 21, 64, e, None) == 2
    assert f(*a, 0, 512, 512, e, None) == 0
    assert f(*a[:6], _vp(FAR + 8), 128, 512, 512, e, None) == 3
    n = L.nvq_linear_epilogue
    w = [_vp(FAR)] * 3
    assert n(_vp(FAR), 1, 256, 512, *w, None, None, -1, _vp(FAKE), e, None, 0, None) == 1
    assert n(_vp(FAR), 64, 256, 512, None, None, None, *w[:2], -1, _vp(FAKE), e, _vp(FAR), 1 << 40, None) == 1
    assert n(_vp(FAR), 64, 256, 512, *w, None, None, -1, _vp(FAKE), e, _vp(FAR), 16, None) == 4
    assert n(_vp(FAR), 64, 256, 512, *w, None, None, -1, _vp(FAKE), e, _vp(ODD), 1 << 40, None) == 3


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        nvq.w4a16_gemm_epilogue(x, x, x, 32)
    with pytest.raises(ValueError, match="CUDA"):
        nvq.nvfp4_gemm_w4a4_epilogue((x, x, x), (x, x, x), 2, 32, 128)
    with pytest.raises(ValueError, match="CUDA"):
        nvq.nvq_linear_epilogue(x, N=32)
