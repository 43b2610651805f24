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
    for kw in (dict(E=513), dict(topk=17), dict(H=192), dict(I=64), dict(H=1 << 20), dict(I=1 << 20), dict(T=1 << 31),
               dict(H=1 << 17, I=1 << 16)):
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


# ------------------------------------------------------------------ mirrors of the kernel's index arithmetic
WARPS, COLS, GRIDS, UNIT_COST = (8, 16), 8, (148, 132), 28


def plan(ids, E):
    """(segments as (expert, first slot, tokens), slot -> pair) as the kernel builds them: up to 32
    pairs by one warp, experts in the order of their first pair; else by token masks, in expert order."""
    T, topk = ids.shape
    flat = [int(v) for v in ids.ravel()]
    first = [0 <= v < E and v not in flat[i // topk * topk:i] for i, v in enumerate(flat)]
    if T * topk <= 32:
        order = []
        for i, v in enumerate(flat):
            if first[i] and v not in order:
                order.append(v)
    else:
        order = range(E)
    segs, pair = [], []
    for e in order:
        mine = [i for i, v in enumerate(flat) if first[i] and v == e]         # by token: the rank is a count of mask bits
        segs += [(e, len(pair) + q, min(COLS, len(mine) - q)) for q in range(0, len(mine), COLS)]
        pair += mine
    return segs, pair


def _random_ids(rng):
    T, topk, E = int(rng.integers(1, 33)), int(rng.integers(1, 17)), int(rng.integers(1, 40))
    return rng.integers(-2, E + 2, size=(T, topk)), E


def test_plan_holds_every_choice_once():
    rng = np.random.default_rng(1)
    for _ in range(300):
        ids, E = _random_ids(rng)
        T, topk = ids.shape
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
        assert [s for _, s, _ in segs] == [sum(n for _, _, n in segs[:i]) for i in range(len(segs))]


def fast_div(d):
    """The kernel's n / d for n < 2^31."""
    l = 0
    while l < 31 and (1 << l) < d:
        l += 1
    mul, shift = ((1 << (31 + l)) + d - 1) // d, 31 + l
    assert mul < 1 << 32
    return lambda n: (n * mul) >> shift


def test_fast_division_is_exact():
    rng = random.Random(4)
    for d in [*range(1, 300), 1 << 16, (1 << 16) + 1, (1 << 20) - 1, 65535, 8192]:
        f = fast_div(d)
        tops = [(1 << 31) - 1, ((1 << 31) - 1) // d * d, ((1 << 31) - 1) // d * d - 1]
        for n in tops + [0, 1, d - 1, d, d + 1] + [rng.randrange(1 << 31) for _ in range(50)]:
            if n >= 0:
                assert f(n) == n // d


def cut(n, w, parts):
    return n * w // parts


def first_tile(segs, rtiles, grid, b, pairs):
    slots = segs[-1][1] + segs[-1][2] if segs else 0
    if pairs <= 32:
        tiles = len(segs) * rtiles
        return b * (tiles // grid) + min(b, tiles % grid)
    cost = (UNIT_COST * len(segs) + slots) * rtiles
    quot, rest = cost // grid, cost % grid
    at = b * quot + min(b, rest)
    s = sum((UNIT_COST * k + seg[1]) * rtiles <= at for k, seg in enumerate(segs))
    if s == 0 or at == cost:
        return len(segs) * rtiles
    s -= 1
    return s * rtiles + (at - (UNIT_COST * s + segs[s][1]) * rtiles) // (UNIT_COST + segs[s][2])


def test_gate_up_split_covers_every_unit_once():
    rng, nrng = random.Random(2), np.random.default_rng(2)
    for _ in range(150):
        ids, E = _random_ids(nrng)
        segs, _ = plan(ids, E)
        warps = rng.choice(WARPS)
        rtiles, G, grid = rng.choice([8, 16, 40, 88]), rng.choice([1, 2, 9, 16, 40]), rng.choice([1, 7, *GRIDS])
        bounds = [first_tile(segs, rtiles, grid, b, ids.size) for b in range(grid + 1)]
        assert bounds == sorted(bounds) and bounds[-1] == len(segs) * rtiles and (not segs or bounds[0] == 0)
        for b in rng.sample(range(grid), min(grid, 6)):
            mine = bounds[b + 1] - bounds[b]
            length = mine * G
            direct, slots = set(), {}
            for w in range(warps):
                f0, f1 = cut(length, w, warps), cut(length, w + 1, warps)
                if f0 == f1:
                    continue
                tile, g, start = f0 // G, f0 % G, f0
                head = g != 0
                for f in range(f0, f1):
                    g += 1
                    if g == G:
                        if head:
                            slots[w, 0] = (tile, start, f + 1)
                        else:
                            direct.add(tile)
                            assert start == tile * G
                        head, g, tile, start = False, 0, tile + 1, f + 1
                if g:
                    slots[w, 0 if f0 // G == (f1 - 1) // G else 1] = (tile, start, f1)
            finished = set()
            for w in range(1, warps):
                f0 = cut(length, w, warps)
                tb = f0 // G * G
                te = tb + G
                if f0 != tb and f0 < length and cut(length, w - 1, warps) <= tb:
                    at, k = tb, w - 1
                    while k < warps and cut(length, k, warps) < te:
                        a = cut(length, k, warps)
                        if a != cut(length, k + 1, warps):
                            tile, s0, s1 = slots.pop((k, 0 if a >= tb else 1))
                            assert tile == tb // G and s0 == at
                            at = s1
                        k += 1
                    assert at == te
                    finished.add(tb // G)
            assert not slots and finished | direct == set(range(mine)) and not finished & direct


def down_cut(U, ntile, grid, b, warps):
    """(half, whole, parts, q, r, F0, F1, n0, n1) of CTA b, of so many warps."""
    total, rounds = U * ntile, -(-U // warps)
    joined = total // warps // grid + (5 if warps == 8 else 4)
    half = 2 * ntile <= grid and rounds * 5 <= joined * 8
    whole = half or -(-ntile // grid) * rounds <= joined
    pieces = (2 * ntile if half else ntile) if whole else total
    parts = min(grid, pieces if whole else -(-total // warps))
    q, r = pieces // parts, pieces % parts
    P0, P1 = b * q + min(b, r), (b + 1) * q + min(b + 1, r)
    k = U if whole else 1
    n0, n1 = (P0 // (U if not whole else 1), (P1 - 1) // (U if not whole else 1)) if b < parts else (1, 0)
    return half, whole, parts, q, r, P0 * k, P1 * k, n0, n1


def test_down_split_covers_every_unit_once_and_finds_every_part():
    rng = random.Random(3)
    modes = set()
    for _ in range(600):
        warps = rng.choice(WARPS)
        grid, ntile, U = rng.choice([2, *GRIDS]), rng.choice([4, 8, 64, 74, 75, 128, 149, 160, 300]), rng.choice([1, 2, 3, 12, 48, 96, 97, 672])
        half, whole_mode, parts, q, r, *_ = down_cut(U, ntile, grid, 0, warps)
        modes.add((half, whole_mode))
        tiles = 2 * ntile if half else ntile
        owner = lambda u: u // (q + 1) if u < r * (q + 1) else r + (u - r * (q + 1)) // q   # noqa: E731
        bound = lambda b: (b * q + min(b, r))                                            # noqa: E731
        count, slot_of, whole, end = {}, {}, set(), 0
        for b in range(grid):
            *_, F0, F1, n0, n1 = down_cut(U, ntile, grid, b, warps)
            if n0 > n1:
                assert b >= parts
                continue
            assert F0 == end and F1 > F0 and n0 == F0 // U and n1 == (F1 - 1) // U
            end, cut_tiles = F1, []
            for n in range(n0, n1 + 1):
                tb = n * U
                if F0 <= tb and F1 >= tb + U:
                    assert n not in whole
                    whole.add(n)
                else:
                    cut_tiles.append(n)
                    count[n] = count.get(n, 0) + 1
                    s = 2 * b + (0 if F0 >= tb else 1)
                    assert s not in slot_of                   # a slot holds one tile's part
                    slot_of[s] = n
                lo = max(F0, tb) - tb
                size = min(F1, tb + U) - tb - lo
                at = lo
                for w in range(warps):                        # the warps' shares follow one another
                    assert lo + size * w // warps == at
                    at = lo + size * (w + 1) // warps
                assert at == lo + size
            assert set(cut_tiles) <= {n0, n1} and not (whole_mode and cut_tiles)
        assert end == tiles * U
        assert whole | set(count) == set(range(tiles)) and not whole & set(count)
        for n, c in count.items():
            tb = n * U
            b0, b1 = owner(tb), owner(tb + U - 1)
            assert b1 - b0 + 1 == c
            for b in range(b0, b1 + 1):
                s = 2 * b + ((0 if bound(b0) >= tb else 1) if b == b0 else 0)
                assert slot_of[s] == n
    assert modes == {(True, True), (False, True), (False, False)}


def h_at(column):
    """Where the kernel keeps a column of h: by row tile and row, as gate and up write it."""
    rt, row = divmod(column, 16)
    k = (rt & 7) * 16
    return (rt >> 3) * 128 + (k & 16) * 4 + (k >> 5) * 8 + (row & 7) + 32 * (row >> 3)


def test_order_of_h_is_the_one_that_down_reads():
    at = [h_at(k) for k in range(512)]
    assert sorted(at) == list(range(512))
    for grp in range(4):
        for c in range(4):
            for i in range(4):
                for e in range(8):                            # lane c's i-th load: 8 values from 32 i + 8 c on
                    assert at[grp * 128 + 32 * c + 8 * i + e] == grp * 128 + 32 * i + 8 * c + e
