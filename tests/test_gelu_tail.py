"""GELU where it is small: z (1 + erf(z / sqrt 2)) / 2 for negative z, whose digits a difference of 1 and erf loses.

Tolerance, relative to the value: half a BF16 step 2^-8; z Phi(z) = z exp(-z^2 / 2) R(|z|), where the
FP32 argument -z^2 / 2 log2(e) has three roundings (z^2, the constant, the product), 1.5 x 2^-23
together, and moves the result by z^2 / 2 of that: below z^2 2^-23.  The fit of R is good to
9.4e-8 < 2^-23, its eight coefficients and steps add less than 2 x 2^-23 (all sums between 0.1 and
0.6), power of two and reciprocal 2 x 2^-23 each (the reciprocal enters R once or twice), the
products 2 x 2^-23: 8 x 2^-23 = 2^-20 at most.
"""
import math

import numpy as np
import pytest
import torch

import phase_disaggregated_quantized_b200 as nvq
from oracle import epilogue as oepi

from helpers import bf16_to_f64

TAIL = [-0.01, -0.5, -1.0, -2.0, -3.0, -4.0, -4.25, -4.5, -4.75, -5.0, -5.25, -5.5, -5.75, -6.0, -7.0, -8.0, -9.0, -10.0,
        -11.0, -12.0, 0.01, 0.5, 1.0, 3.0, 4.5, 5.5, 6.0, 12.0, 1e10, 0.0, -0.0, 100.0]
N = len(TAIL)                                                # 32


def _tolerance(z, want):
    return (2.0 ** -8 + np.minimum(z * z + 1, 200) * 2.0 ** -23 + 2.0 ** -20) * np.abs(want)


def test_oracle_keeps_the_tail():
    """Against the asymptotic series of Mills' ratio: gelu(z) = -phi(z) (1 - 1/z^2 + 3/z^4 - 15/z^6 + 105/z^8 - ...), alternating."""
    for z in (-6.0, -8.0, -12.0):
        phi = math.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        upper = -phi * (1 - z ** -2 + 3 * z ** -4 - 15 * z ** -6 + 105 * z ** -8 - 945 * z ** -10)
        lower = -phi * (1 - z ** -2 + 3 * z ** -4 - 15 * z ** -6 + 105 * z ** -8)
        assert lower <= oepi.activation(np.array([z]), "gelu")[0] <= upper
    with np.errstate(invalid="ignore"):
        assert oepi.activation(np.array([np.inf]), "gelu")[0] == np.inf and np.isnan(oepi.activation(np.array([np.nan]), "gelu")[0])


@pytest.mark.gpu
@pytest.mark.parametrize("form, M", [("w4a16", 2), ("w4a16", 20), ("w4a4", 2), ("w4a4", 40000)])
def test_gelu_keeps_its_tail(form, M):
    """x of all zeros: y = gelu(bias).  Every epilogue that computes it: the streaming and the tensor-memory
    INT4 product, the NVFP4 product with its tile split over CTAs and with more tiles than SMs."""
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    z = torch.tensor(TAIL).to(torch.bfloat16)
    x = torch.zeros(M, 128, dtype=torch.bfloat16, device="cuda")
    w = torch.randn(N, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    if form == "w4a16":
        y = nvq.w4a16_gemm_epilogue(x, *nvq.int4_pack_weights(*nvq.int4_quantize(w), N, 128), N, bias=z.cuda(), activation="gelu")
    else:
        y = nvq.nvfp4_gemm_w4a4_epilogue(nvq.nvfp4_quantize(x), nvq.nvfp4_quantize(w), M, N, 128, bias=z.cuda(), activation="gelu")
    nvq.check_device_error()
    assert (y == y[0]).all()
    y, zz = bf16_to_f64(y[0]), bf16_to_f64(z)
    want = oepi.activation(zz, "gelu")
    off = np.abs(y - want)
    assert (off <= _tolerance(zz, want)).all(), [(a, b, c) for a, b, c, d in zip(zz, y, want, off > _tolerance(zz, want)) if d]
