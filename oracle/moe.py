"""CPU oracle for the mixture-of-experts layer of a few tokens.

TEST INFRASTRUCTURE ONLY.  Only ``tests/``, ``__graft_entry__.smoke()`` and the
CPU-baseline / reference legs of ``bench.py`` may import this module.  It shares
no code with the CUDA path.

    logits = x Wr^T; ids: the topk largest of a token (ties: the lower index, NaN above numbers);
    weights = exp(l) / sum of exp(l) over the chosen (renormalize) or all experts;
    y = residual + sum_j weights_j Wd[e_j] (silu(Wg[e_j] x) * (Wu[e_j] x))

all in float64.  ``experts`` also returns a bound on what the kernels' arithmetic
may differ by, from these facts (u = 2^-23 is taken for every FP32 operation,
which covers tensor-core additions that truncate):

  * a product of K codes is formed as sum x (code - 8), exact products, and scaled per
    group of 128, partial sums at most A = 8 sum_k |x_k| s_group: at most 8 additions
    within a group, K / 128 over the groups, 16 over warps and 148 over CTAs, so it is
    off by at most d(K) u A with d(K) = 172 + K / 128;
  * h = w silu(g) u with |silu'| <= 1.1: off by |w| (1.1 e_g |u| + |silu(g)| e_u +
    1.1 e_g e_u) + 1e-5 |h| (fast exponential and reciprocal) + 2^-16 |h| (two BF16
    numbers, each rounding at most half a step of 2^-7);
  * down: |Wd| e_h summed, its own additions d(I topk) u over A' = 8 sum |h| s, and the
    residual;
  * one rounding to BF16: 2^-8 |y|.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -23


def silu(z):
    with np.errstate(over="ignore"):
        return z / (1 + np.exp(-z))


def route(x: np.ndarray, wr: np.ndarray, topk: int, renormalize: bool):
    """(ids int32, weights, logits) in float64."""
    logits = x @ wr.T
    key = np.where(np.isnan(logits), np.inf, logits)
    isnan = np.isnan(logits)
    ids = np.zeros((x.shape[0], topk), dtype=np.int32)
    for t in range(x.shape[0]):
        order = sorted(range(wr.shape[0]), key=lambda e: (not isnan[t, e], -key[t, e], e))
        ids[t] = order[:topk]
    with np.errstate(invalid="ignore", over="ignore"):
        l = np.take_along_axis(logits, ids.astype(np.int64), axis=1)
        e = np.exp(l - l[:, :1])
        total = e.sum(1) if renormalize else np.exp(logits - l[:, :1]).sum(1)
        return ids, e / total[:, None], logits


def experts(x, ids, weights, gate, up, down, gate_s, up_s, down_s, residual=None):
    """(y, tolerance).  gate / up [E, I, H], down [E, H, I]: dequantized weights;
    *_s: the group scale of every weight, same shapes."""
    T, H = x.shape
    E, I, _ = gate.shape
    y = np.zeros((T, H)) if residual is None else residual.astype(np.float64).copy()
    tol = U * np.abs(y)
    topk = ids.shape[1]
    d = lambda K: 172 + K / 128                                                     # noqa: E731
    for t in range(T):
        for j in range(topk):
            e = int(ids[t, j])
            if not 0 <= e < E:
                continue
            g, u = gate[e] @ x[t], up[e] @ x[t]
            eg = d(H) * U * 8 * (gate_s[e] @ np.abs(x[t]))
            eu = d(H) * U * 8 * (up_s[e] @ np.abs(x[t]))
            w, sg = float(weights[t, j]), silu(g)
            h = w * sg * u
            eh = abs(w) * (1.1 * eg * np.abs(u) + np.abs(sg) * eu + 1.1 * eg * eu) + (1e-5 + 2.0 ** -16) * np.abs(h)
            y[t] += down[e] @ h
            tol[t] += np.abs(down[e]) @ eh + d(I * topk) * U * 8 * (down_s[e] @ (np.abs(h) + eh))
    return y, tol + 2.0 ** -8 * (np.abs(y) + tol)
