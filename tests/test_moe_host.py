"""The mixture-of-experts layer without a GPU: its oracle, the refusals of the
entry points, and a mirror of how the expert kernels cut and sort their work."""
import ctypes
import random

import numpy as np
import pytest
import torch

import phase_disaggregated_quantized_b200 as nvq
from phase_disaggregated_quantized_b200 import build_lib
from oracle import moe as omoe

FAKE = 0x7F0000000000
FAR = FAKE + (1 << 40)


def _vp(v):
    return ctypes.c_void_p(v)


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return nvq.lib()


# ------------------------------------------------------------------ oracle
def test_route_oracle_by_hand():
    wr = np.array([[1.0, 0], [0, 1], [1, 0], [0.5, 0.5]])
    ids, w, _ = omoe.route(np.array([[2.0, 1.0]]), wr, 3, True)
    assert ids.tolist() == [[0, 2, 3]]                       # 2, 2 (tie: lower index first), 1.5
    e = np.exp([0, 0, -0.5])
    np.testing.assert_allclose(w[0], e / e.sum(), rtol=1e-15)
    _, w, _ = omoe.route(np.array([[2.0, 1.0]]), wr, 1, False)
    np.testing.assert_allclose(w[0, 0], 1 / (2 + np.exp(-1) + np.exp(-0.5)), rtol=1e-15)
    ids, w, _ = omoe.route(np.array([[np.nan, 1.0]]), wr, 2, True)
    assert ids.tolist() == [[0, 1]] and np.isnan(w).all()    # every logit NaN (0 * NaN too)


def test_experts_oracle_by_brute_force():
    rng = np.random.default_rng(0)
    T, E, H, I = 3, 4, 6, 5
    x, g, u, d = rng.normal(size=(T, H)), rng.normal(size=(E, I, H)), rng.normal(size=(E, I, H)), rng.normal(size=(E, H, I))
    ids = np.array([[0, 3], [2, 2], [-1, 9]], dtype=np.int32)
    w = rng.random((T, 2))
    one = np.ones
    y, _ = omoe.experts(x, ids, w, g, u, d, one(g.shape), one(u.shape), one(d.shape))
    for t in range(T):
        for n in range(H):
            s = 0.0
            for j in range(2):
                e = ids[t, j]
                if 0 <= e < E:
                    for i in range(I):
                        a = sum(g[e, i, k] * x[t, k] for k in range(H))
                        b = sum(u[e, i, k] * x[t, k] for k in range(H))
                        s += w[t, j] * d[e, n, i] * a / (1 + np.exp(-a)) * b
            assert y[t, n] == pytest.approx(s, abs=1e-12)
    assert not y[2].any()


# ------------------------------------------------------------------ refusals
def test_route_refuses(L):
    f = L.moe_route
    ok = [_vp(FAKE), _vp(FAKE)]
    out = [1, _vp(FAKE), _vp(FAKE), None]
    assert f(*ok, 0, 8, 128, 2, *out) == 0
    assert f(*ok, -1, 8, 128, 2, *out) == 1
    assert f(*ok, 4, 0, 128, 2, *out) == 1
    assert f(*ok, 4, 8, 0, 2, *out) == 1
    assert f(*ok, 4, 8, 128, 0, *out) == 1
    assert f(*ok, 4, 8, 128, 9, *out) == 1                    # topk > E
    assert f(*ok, 4, 513, 128, 2, *out) == 2
    assert f(*ok, 4, 64, 128, 17, *out) == 2
    assert f(*ok, 4, 8, 96, 2, *out) == 2                     # H % 64
    assert f(*ok, 1 << 31, 8, 128, 2, *out) == 2
    assert f(None, _vp(FAKE), 4, 8, 128, 2, *out) == 1
    assert f(_vp(FAKE + 8), _vp(FAKE), 4, 8, 128, 2, *out) == 3
    assert f(*ok, 4, 8, 128, 2, 1, _vp(FAKE + 2), _vp(FAKE), None) == 3


def _experts(L, T=4, E=8, H=256, I=128, topk=2, x=FAKE, y=FAR, res=None, ws=FAR + (1 << 30), n=1 << 30, null=None, odd=None):
    p = [x, FAKE, FAKE, FAR, FAR, FAR, FAR, res, y]
    if null is not None:
        p[null] = None
    if odd is not None:
        p[odd] += 2
    return L.w4a16_moe_experts(*[_vp(v) for v in p], T, E, H, I, topk, _vp(ws), n, None)


def test_experts_refuse(L):
    assert _experts(L, T=0) == 0
    for kw in (dict(T=-1), dict(E=0), dict(H=0), dict(I=-128), dict(topk=0)):
        assert _experts(L, **kw) == 1, kw
    for kw in (dict(E=513), dict(topk=17), dict(H=192), dict(I=64), dict(H=1 << 20), dict(I=1 << 20), dict(T=1 << 31)):
        assert _experts(L, **kw) == 2, kw
    for i in (0, 1, 2, 3, 4, 5, 6, 8):
        assert _experts(L, null=i) == 1, i
        assert _experts(L, odd=i) == 3, i
    assert _experts(L, res=FAR + (1 << 20) + 2) == 3
    assert _experts(L, y=FAKE + 512) == 1                       # a later row of x
    assert _experts(L, res=FAR + 512) == 1                      # a later row of y
    need = L.w4a16_moe_workspace_bytes(4, 256, 128, 2)
    assert _experts(L, n=need - 1) == 4 and _experts(L, ws=None) == 4
    assert _experts(L, ws=FAR + 8) == 3
    for bad in ((0, 256, 128, 2), (4, 0, 128, 2), (4, 256, 1 << 20, 2), (4, 256, 128, 17)):
        assert L.w4a16_moe_workspace_bytes(*bad) == 0
    assert L.w4a16_moe_workspace_bytes(32, 256, 128, 2) == L.w4a16_moe_workspace_bytes(500, 256, 128, 2) > need


def test_whole_layer_refuses_what_its_parts_refuse(L):
    def call(T=4, E=8, H=256, I=128, topk=2, n=1 << 30, y=FAR):
        return L.w4a16_moe(*[_vp(v) for v in (FAKE, FAKE, FAR, FAR, FAR, FAR, None, y, FAKE, FAKE)], T, E, H, I, topk, 1,
                           _vp(FAR + (1 << 30)), n, None)
    assert call(T=0) == 0
    assert call(topk=9) == 1 and call(H=192) == 2 and call(I=64) == 2 and call(n=16) == 4 and call(y=FAKE + 512) == 1


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        nvq.moe_route(x, x, 1)
    with pytest.raises(ValueError, match="CUDA"):
        nvq.w4a16_moe_experts(x, x, x, (x, x), (x, x), 2, 128)
    with pytest.raises(ValueError, match="CUDA"):
        nvq.w4a16_moe(x, x, (x, x), (x, x), 128, 1)


def test_interleave_in_blocks_of_16():
    g, u = torch.arange(32).view(32, 1).float(), 100 + torch.arange(32).view(32, 1).float()
    w = nvq.interleave_gate_up(g, u, block=16).flatten().tolist()
    assert w == [*range(16), *range(100, 116), *range(16, 32), *range(116, 132)]


# ------------------------------------------------------------------ mirrors of the kernels' index arithmetic
WARPS, COLS = 8, 8


def plan(ids, E):
    """(segments as (expert, first slot, tokens), slot -> pair) as the kernels build them, by masks."""
    T, topk = ids.shape
    first = [[0 <= ids[t, j] < E and ids[t, j] not in ids[t, :j] for j in range(topk)] for t in range(T)]
    mask = [0] * E
    for t in range(T):
        for j in range(topk):
            if first[t][j]:
                mask[ids[t, j]] |= 1 << t
    segs, start, slot = [], {}, 0
    for e in range(E):
        n = bin(mask[e]).count("1")
        start[e] = slot
        segs += [(e, slot + q, min(COLS, n - q)) for q in range(0, n, COLS)]
        slot += n
    pair = [None] * slot
    for t in range(T):
        for j in range(topk):
            if first[t][j]:
                e = ids[t, j]
                pair[start[e] + bin(mask[e] & ((1 << t) - 1)).count("1")] = t * topk + j
    return segs, pair


def test_plan_holds_every_choice_once():
    rng = np.random.default_rng(1)
    for _ in range(300):
        T, topk, E = int(rng.integers(1, 33)), int(rng.integers(1, 17)), int(rng.integers(1, 40))
        ids = rng.integers(-2, E + 2, size=(T, topk))
        segs, pair = plan(ids, E)
        want = sorted({(int(ids[t, j]), t) for t in range(T) for j in range(topk) if 0 <= ids[t, j] < E})
        got = []
        for e, s, n in segs:
            toks = [pair[k] // topk for k in range(s, s + n)]
            assert 1 <= n <= COLS and len(set(toks)) == n
            assert all(ids[pair[k] // topk, pair[k] % topk] == e for k in range(s, s + n))
            got += [(e, t) for t in toks]
        assert sorted(got) == want
        assert len(segs) <= T * topk


def cut(n, w, parts):
    return n * w // parts


def test_gate_up_split_covers_every_unit_once():
    rng = random.Random(2)
    for _ in range(400):
        grid, tiles, G = rng.choice([1, 7, 296]), rng.choice([0, 1, 3, 50, 400, 5000]), rng.choice([1, 2, 9, 16, 40])
        for b in rng.sample(range(grid), min(grid, 8)):
            T0, T1 = cut(tiles, b, grid), cut(tiles, b + 1, grid)
            length = (T1 - T0) * G
            direct, slots = set(), {}
            for w in range(WARPS):
                f0, f1 = cut(length, w, WARPS), cut(length, w + 1, WARPS)
                if f0 == f1:
                    continue
                tile, g, start = f0 // G, f0 % G, f0
                for f in range(f0, f1):
                    g += 1
                    if g == G:
                        if f0 % G and tile == f0 // G:
                            slots[w, 0] = (tile, start, f + 1)
                        else:
                            direct.add(tile)
                            assert start == tile * G and f + 1 == start + G
                        g, tile, start = 0, tile + 1, f + 1
                if g:
                    slots[w, 0 if tile == f0 // G else 1] = (tile, start, f1)
            for i in range(T1 - T0):
                tb, te = i * G, (i + 1) * G
                at = tb
                for w in range(WARPS):
                    a, e = cut(length, w, WARPS), cut(length, w + 1, WARPS)
                    if a < e and a < te and e > tb and not (a <= tb and e >= te):
                        tile, s0, s1 = slots.pop((w, 0 if a >= tb else 1))
                        assert tile == i and s0 == at
                        at = s1
                assert at in (tb, te) and (i in direct) == (at == tb)
            assert not slots


def test_down_split_covers_every_unit_once_and_finds_every_part():
    rng = random.Random(3)
    for _ in range(400):
        grid, tiles, U = rng.choice([2, 296]), rng.choice([4, 8, 64, 160]), rng.choice([1, 2, 3, 12, 48, 672])
        total = tiles * U
        parts = min(grid, -(-total // WARPS))
        seen, count, slot_of = 0, {}, {}
        for b in range(parts):
            F0, F1 = total * b // parts, total * (b + 1) // parts
            assert F0 == seen and F1 > F0
            seen = F1
            n = F0 // U
            while n * U < F1:
                tb, te = n * U, n * U + U
                if not (F0 <= tb and F1 >= te):
                    count[n] = count.get(n, 0) + 1
                    s = 2 * b + (0 if F0 >= tb else 1)
                    assert s not in slot_of                   # a slot holds one tile's part
                    slot_of[s] = n
                n += 1
        assert seen == total
        for n, c in count.items():
            tb, te = n * U, n * U + U
            b0, b1 = ((tb + 1) * parts - 1) // total, (te * parts - 1) // total
            assert b1 - b0 + 1 == c
            for b in range(b0, b1 + 1):
                assert slot_of[2 * b + (0 if total * b // parts >= tb else 1)] == n
