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


# ------------------------------------------------------------------ the work split of the INT4 product with more than 8 rows
def tmem_split(tiles, G):
    """(log2 of the CTAs per cluster, rounds of whole tiles, clusters), as the host chooses them."""
    at_once, end, best, least = (148, 74, 33, 15), (6, 15, 18, 24), None, 1 << 62
    for l in range(4):
        if (1 << l) > G:
            break
        one, shared, ctas = 2 * G + end[0], 2 * -(-G // (1 << l)) + end[l], at_once[l] << l
        rounds = -(-tiles // at_once[l])
        if rounds * shared < least:
            best, least = (l, 0, -(-tiles // rounds)), rounds * shared
        solo = tiles // ctas if l else 0
        cost = solo * one + -(-(tiles - solo * ctas) // at_once[l]) * shared
        if solo and cost < least:
            best, least = (l, solo, at_once[l]), cost
    return best


@pytest.mark.parametrize("tiles", [1, 2, 15, 16, 33, 34, 74, 75, 99, 148, 149, 150, 192, 223, 296, 297, 700])
@pytest.mark.parametrize("G", [1, 2, 3, 7, 8, 32, 48, 128, 400])
def test_int4_jobs_cover_every_tile_and_group_once(tiles, G):
    slog, solo, clusters = tmem_split(tiles, G)
    slices = 1 << slog
    seen = {}
    for cid in range(clusters):
        first = solo * (clusters << slog) + cid
        jobs = solo + ((tiles - 1 - first) // clusters + 1 if first < tiles else 0)
        assert jobs >= 1
        for rank in range(slices):
            for j in range(jobs):
                whole = j < solo
                tile = (j * clusters + cid) * slices + rank if whole else first + (j - solo) * clusters
                k0, k1 = (0, G) if whole else (G * rank >> slog, G * (rank + 1) >> slog)
                assert 0 <= tile < tiles and k0 < k1
                seen.setdefault(tile, []).append((k0, k1))
    assert sorted(seen) == list(range(tiles))
    for parts in seen.values():
        parts.sort()
        assert parts[0][0] == 0 and parts[-1][1] == G and all(a[1] == b[0] for a, b in zip(parts, parts[1:]))
