"""CPU oracle for the products with bias, activation and residual in their epilogue.

TEST INFRASTRUCTURE ONLY.  Only ``tests/``, ``__graft_entry__.smoke()`` and the
CPU-baseline / reference legs of ``bench.py`` may import this module.  It shares
no code with the CUDA path.

    y = act(v + bias) + residual        (float64; v the exact product)

The comparison.  The kernels hold v, the bias sum, the activation and the
residual sum in FP32 and round once to BF16.  With |v_gpu - v| <= e, where
e = 1e-3 rms(v) + 1e-5 |v| bounds the FP32 accumulation (the library's bar for a
product without its BF16 rounding), the result differs from y by at most

    L e  +  1e-5 |act|  +  2^-23 (|z| + |act| + |y|)  +  2^-8 |y + those|

L = 1.13 bounds |act'| of every activation here (gelu: 1.1290, gelu_tanh:
1.1290, silu: 1.0998), 1e-5 |act| covers the fast exponential and reciprocal, the
2^-23 terms the FP32 sums, and 2^-8 |.| half a BF16 step.
"""
from __future__ import annotations

import math

import numpy as np

ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")
MAX_SLOPE = 1.13

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def activation(z: np.ndarray, name: str) -> np.ndarray:
    z = np.asarray(z, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if name == "none":
            return z
        if name == "relu":
            return np.where(z < 0, 0.0, z)
        if name == "gelu":
            return 0.5 * z * _erfc(-z / math.sqrt(2))             # 1 + erf(u) = erfc(-u), without its cancellation
        if name == "gelu_tanh":
            return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
        if name == "silu":
            return z / (1 + np.exp(-z))
    raise ValueError(name)


def apply(v: np.ndarray, bias=None, act: str = "none", residual=None):
    """(y, tolerance) of a product v in float64."""
    v = np.asarray(v, dtype=np.float64)
    z = v if bias is None else v + bias
    a = activation(z, act)
    y = a if residual is None else a + residual
    e = 1e-3 * np.sqrt(np.mean(v * v)) + 1e-5 * np.abs(v)
    tol = MAX_SLOPE * e + 1e-5 * np.abs(a) + 2.0 ** -23 * (np.abs(z) + np.abs(a) + np.abs(y))
    return y, tol + 2.0 ** -8 * (np.abs(y) + tol)
