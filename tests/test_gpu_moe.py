"""The mixture-of-experts layer on the GPU against the float64 oracle.

Tolerances: oracle.moe.experts (its docstring derives them); the router's
logits: each MMA adds 16 exact products (at most 16 truncations at 2^-23 of the
sum of magnitudes S), then at most H / 64 + 16 + 4 FP32 sums, so a logit is off by
at most dl = (36 + H / 64) 2^-23 S; a weight by a relative 2 dl + 2^-20 (exp, sum
of at most 512 terms in a tree, division).
"""
import numpy as np
import pytest
import torch

import phase_disaggregated_quantized_b200 as nvq
from phase_disaggregated_quantized_b200 import synth
from oracle import int4 as oint4
from oracle import moe as omoe

from helpers import bf16_to_f64, oracle_int4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from phase_disaggregated_quantized_b200 import build_lib
    build_lib.build()
    nvq.lib()
    yield
    nvq.check_device_error()


# ------------------------------------------------------------------ router
def _check_route(x, wr, topk, renorm, ids, weights):
    X, W = bf16_to_f64(x), bf16_to_f64(wr)
    want, ww, logits = omoe.route(X, W, topk, renorm)
    dl = (36 + X.shape[1] / 64) * 2.0 ** -23 * (np.abs(X) @ np.abs(W).T).max(1)
    ids, weights = ids.cpu().numpy(), weights.cpu().numpy().astype(np.float64)
    got = np.take_along_axis(logits, ids.astype(np.int64), 1)
    ref = np.take_along_axis(logits, want.astype(np.int64), 1)
    assert all(len(set(r)) == topk for r in ids)
    assert (np.abs(got - ref) <= 2 * dl[:, None]).all()                # the j-th choice has the j-th logit
    same = ids == want
    assert same.mean() > 0.99                                         # and is the same expert but for near ties
    rel = np.abs(weights - ww) / ww
    assert (rel[same] <= np.broadcast_to((2 * dl + 2.0 ** -20)[:, None], rel.shape)[same]).all(), rel[same].max()


@pytest.mark.parametrize("T, E, H, topk", [
    (1, 1, 64, 1), (1, 128, 4096, 8), (2, 2, 128, 2), (5, 17, 192, 16), (8, 60, 2048, 4), (31, 128, 704, 8),
    (32, 384, 1024, 6), (33, 512, 256, 16), (56, 200, 640, 3), (64, 16, 512, 1), (70, 8, 8192, 2), (3, 257, 320, 5), (113, 130, 192, 4),
    (300, 512, 128, 2)])
def test_route_matches_the_oracle(T, E, H, topk):
    g = torch.Generator().manual_seed(T + E + H)
    x = synth.activations(T, H, seed=T)
    wr = (torch.randn(E, H, generator=g) * 0.05).to(torch.bfloat16)
    for renorm in (True, False):
        ids, w = nvq.moe_route(x.cuda(), wr.cuda(), topk, renormalize=renorm)
        assert ids.dtype == torch.int32 and w.dtype == torch.float32
        _check_route(x, wr, topk, renorm, ids, w)
    assert nvq.moe_route(x.cuda()[:0], wr.cuda(), topk)[0].shape == (0, topk)


def test_route_ties_go_to_the_lower_index():
    x = torch.randn(9, 256, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    wr = torch.randn(4, 256, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).repeat(24, 1)   # 24 copies of 4
    ids, w = nvq.moe_route(x.cuda(), wr.cuda(), 10)
    first = omoe.route(bf16_to_f64(x), bf16_to_f64(wr[:4]), 1, True)[0][:, 0]
    assert ids.cpu().tolist() == [[int(f) + 4 * j for j in range(10)] for f in first]
    assert (w == w[0, 0]).all()
    ids, w = nvq.moe_route(torch.zeros_like(x).cuda(), wr.cuda(), 3, renormalize=False)       # all logits 0
    assert (ids.cpu() == torch.arange(3)).all() and torch.allclose(w.cpu(), torch.full((9, 3), 1 / 96), rtol=1e-6)
    neg = -torch.zeros_like(x)                                                          # all logits -0 or +0
    assert (nvq.moe_route(neg.cuda(), wr.cuda(), 3)[0].cpu() == torch.arange(3)).all()


def test_route_values_that_are_not_finite():
    x = torch.ones(3, 64, dtype=torch.bfloat16)
    x[1] = float("nan")
    wr = torch.full((40, 64), 0.25, dtype=torch.bfloat16)
    wr[7], wr[33] = float("nan"), float("-inf")
    ids, w = nvq.moe_route(x.cuda(), wr.cuda(), 3)
    assert ids.cpu().tolist() == [[7, 0, 1], [0, 1, 2], [7, 0, 1]]
    assert torch.isnan(w).all()
    wr[7] = 0.25
    ids, w = nvq.moe_route(x[:1].cuda(), wr.cuda(), 16, renormalize=False)
    assert ids.cpu().tolist() == [list(range(16))]
    assert torch.allclose(w.cpu(), torch.full((1, 16), 1 / 39), rtol=1e-6)              # exp(-inf) = 0
    wr[:] = float("-inf")
    ids, _ = nvq.moe_route(x[:1].cuda(), wr.cuda(), 16)
    assert ids.cpu().tolist() == [list(range(16))]


# ------------------------------------------------------------------ experts
class Layer:
    def __init__(self, E, H, I, seed=0):
        self.E, self.H, self.I = E, H, I
        g = torch.Generator().manual_seed(seed)
        draw = lambda *s: (torch.randn(*s, generator=g) * 0.05).to(torch.bfloat16)                 # noqa: E731
        gate, up, down = draw(E, I, H), draw(E, I, H), draw(E, H, I)
        gu = torch.cat([nvq.interleave_gate_up(gate[e], up[e], block=16) for e in range(E)])
        self.gate_up = self._pack(gu)
        self.down = self._pack(down.view(E * H, I))
        self.parts = []
        for w in (gate, up, down):
            u, s = oracle_int4(w.reshape(-1, w.shape[2]))
            val = oint4.dequantize(u, s).reshape(w.shape)
            sc = np.repeat(oint4.bf16_bits_to_f64(s), 128, axis=1).reshape(w.shape)
            self.parts.append((val, sc))

    @staticmethod
    def _pack(w):
        c, s = nvq.int4_quantize(w.cuda())
        return nvq.int4_pack_weights(c, s, *w.shape)

    def __call__(self, x, ids, weights, **kw):
        return nvq.w4a16_moe_experts(x, ids, weights, self.gate_up, self.down, self.E, self.I, **kw)

    def oracle(self, x, ids, weights, residual=None):
        (g, gs), (u, us), (d, ds) = self.parts
        return omoe.experts(bf16_to_f64(x), ids.cpu().numpy(), weights.cpu().double().numpy(), g, u, d, gs, us, ds,
                            None if residual is None else bf16_to_f64(residual))


def _choices(T, E, topk, seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(E, generator=g)[:topk] for _ in range(T)]).to(torch.int32)
    return ids, torch.softmax(torch.randn(T, topk, generator=g), 1)


def _check(y, want, tol):
    off = np.abs(bf16_to_f64(y) - want)
    assert (off <= tol).all(), f"worst {np.nanmax(off / tol):.3f} of the tolerance"


_LAYERS = {}


def layer(E, H, I):
    if (E, H, I) not in _LAYERS:
        _LAYERS[E, H, I] = Layer(E, H, I, seed=E + H + I)
    return _LAYERS[E, H, I]


@pytest.mark.parametrize("T, E, H, I, topk", [
    (1, 1, 128, 128, 1), (1, 8, 256, 128, 2), (1, 40, 128, 384, 8), (2, 3, 640, 256, 3), (7, 8, 384, 128, 2),
    (8, 2, 256, 256, 1), (9, 2, 256, 256, 2), (17, 1, 128, 256, 1), (31, 5, 256, 384, 4), (32, 16, 128, 128, 16),
    (32, 40, 128, 384, 8), (33, 8, 256, 128, 2), (70, 3, 640, 256, 2), (32, 512, 128, 128, 3),
    # more weights than two units per warp of small CTAs: sixteen warps, every way of cutting the down phase
    (1, 8, 4096, 512, 4), (3, 24, 640, 1408, 8), (32, 24, 896, 640, 4), (20, 48, 384, 1536, 16), (40, 6, 2048, 768, 2), (32, 4, 4096, 1280, 2),
    # very long rows of x
    (1, 1, 65664, 128, 1), (5, 2, 65664, 128, 1)])
def test_experts_match_the_oracle(T, E, H, I, topk):
    lay = layer(E, H, I)
    x = synth.activations(T, H, seed=T)
    ids, w = _choices(T, E, topk, T)
    res = torch.randn(T, H, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16)
    for r in (None, res):
        y = lay(x.cuda(), ids.cuda(), w.cuda(), residual=None if r is None else r.cuda())
        nvq.check_device_error()
        _check(y, *lay.oracle(x, ids, w, r))


@pytest.mark.parametrize("T", [4, 8, 12, 16, 24, 32])
def test_every_token_at_the_same_experts(T):
    lay = layer(8, 256, 128)
    x = synth.activations(T, 256, seed=T)
    ids = torch.tensor([[5, 2]], dtype=torch.int32).repeat(T, 1)
    w = torch.rand(T, 2, generator=torch.Generator().manual_seed(T))
    _check(lay(x.cuda(), ids.cuda(), w.cuda()), *lay.oracle(x, ids, w))


def test_rows_without_a_choice_and_ids_out_of_range():
    """Padded rows hold NaN and no id: they get their residual (or 0), nobody else sees them."""
    lay = layer(8, 256, 128)
    x = synth.activations(12, 256, seed=2)
    ids, w = _choices(12, 8, 2, 2)
    x[9:] = float("nan")
    ids[9], ids[10], ids[11] = -1, torch.tensor([8, 2 ** 31 - 1], dtype=torch.int32), torch.tensor([-2 ** 31, 9], dtype=torch.int32)
    w[9:] = float("nan")
    ids[0, 1], ids[1] = -1, 8
    res = torch.randn(12, 256, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    y = lay(x.cuda(), ids.cuda(), w.cuda(), residual=res.cuda())
    for rows in (slice(1, 2), slice(9, 12)):
        assert torch.equal(y[rows].cpu(), res[rows])
    keep = [0, *range(2, 9)]
    _check(y[keep], *lay.oracle(x[keep], ids[keep], w[keep], res[keep]))
    none = torch.full_like(ids, -1)
    assert torch.equal(lay(x.cuda(), none.cuda(), w.cuda(), residual=res.cuda()).cpu(), res)
    assert not lay(x.cuda(), none.cuda(), w.cuda(), y=torch.ones(12, 256, dtype=torch.bfloat16, device="cuda")).any()
    assert lay(x.cuda()[:0], ids.cuda()[:0], w.cuda()[:0]).shape == (0, 256)


def test_an_expert_named_twice_counts_with_both_weights():
    lay = layer(8, 256, 128)
    x = synth.activations(11, 256, seed=4)
    ids = torch.randint(0, 3, (11, 5), generator=torch.Generator().manual_seed(4)).to(torch.int32)
    w = torch.rand(11, 5, generator=torch.Generator().manual_seed(5))
    _check(lay(x.cuda(), ids.cuda(), w.cuda()), *lay.oracle(x, ids, w))


def test_a_token_with_nan_leaves_the_others_alone():
    lay = layer(8, 256, 128)
    x = synth.activations(10, 256, seed=6)
    ids = torch.tensor([[1, 3]], dtype=torch.int32).repeat(10, 1)
    w = torch.rand(10, 2, generator=torch.Generator().manual_seed(6))
    clean = lay(x.cuda(), ids.cuda(), w.cuda())
    x[4, 17] = float("nan")
    y = lay(x.cuda(), ids.cuda(), w.cuda())
    keep = [i for i in range(10) if i != 4]
    assert torch.isnan(y[4].float()).all() and torch.equal(y[keep], clean[keep])


def test_h_keeps_more_than_one_bf16():
    """The error is that of rounding y once: carrying h in one BF16 would add as much again (a factor 1.4)."""
    E, H, I, T = 2, 1024, 1024, 32
    lay = layer(E, H, I)
    x = synth.activations(T, H, seed=7)
    ids, w = _choices(T, E, 2, 7)
    y = bf16_to_f64(lay(x.cuda(), ids.cuda(), w.cuda()))
    want, _ = lay.oracle(x, ids, w)
    rounded = torch.from_numpy(want).to(torch.bfloat16).double().numpy()
    assert np.linalg.norm(y - want) <= 1.1 * np.linalg.norm(rounded - want)


@pytest.mark.parametrize("T", [1, 20, 50])
def test_y_may_be_x_or_the_residual(T):
    lay = layer(8, 256, 128)
    x = synth.activations(T, 256, seed=8).cuda()
    ids, w = (t.cuda() for t in _choices(T, 8, 2, 8))
    res = torch.randn(T, 256, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    want = lay(x, ids, w, residual=res)
    stream, copy = res.clone(), x.clone()
    assert lay(x, ids, w, residual=stream, y=stream) is stream and torch.equal(stream, want)
    assert torch.equal(lay(copy, ids, w, residual=res, y=copy), want)
    both = x.clone()
    assert torch.equal(lay(both, ids, w, residual=both, y=both), lay(x, ids, w, residual=x))


def test_workspace_of_any_content_and_nothing_behind_it():
    lay = layer(40, 128, 384)
    T, topk = 32, 8
    x = synth.activations(T, 128, seed=9).cuda()
    ids, w = (t.cuda() for t in _choices(T, 40, topk, 9))
    want = lay(x, ids, w)
    need = nvq.w4a16_moe_workspace_bytes(T, 128, 384, topk)
    buf = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        y = torch.full((T + 1, 128), 9.0, dtype=torch.bfloat16, device="cuda")
        lay(x, ids, w, workspace=buf[:need], y=y[:T])
        assert torch.equal(y[:T], want) and (y[T] == 9).all() and (buf[need:] == 255).all()
    with pytest.raises(nvq.NvqError, match="workspace"):
        lay(x, ids, w, workspace=buf[:need - 16])


def test_whole_layer_is_its_two_parts():
    lay = layer(40, 128, 384)
    g = torch.Generator().manual_seed(10)
    wr = (torch.randn(40, 128, generator=g) * 0.1).to(torch.bfloat16).cuda()
    for T in (1, 5, 32, 40):
        for renorm in (True, False):
            x = synth.activations(T, 128, seed=T).cuda()
            ids, w = nvq.moe_route(x, wr, 8, renormalize=renorm)
            y, i2, w2 = nvq.w4a16_moe(x, wr, lay.gate_up, lay.down, 384, 8, renormalize=renorm, residual=x)
            assert torch.equal(i2, ids) and torch.equal(w2, w) and torch.equal(y, lay(x, ids, w, residual=x))


def test_repeated_and_concurrent_calls_agree():
    lay = layer(40, 128, 384)
    wr = (torch.randn(40, 128, generator=torch.Generator().manual_seed(11)) * 0.1).to(torch.bfloat16).cuda()
    xs = [synth.activations(T, 128, seed=T).cuda() for T in (3, 32)]
    run = lambda x, **kw: nvq.w4a16_moe(x, wr, lay.gate_up, lay.down, 384, 8, **kw)                # noqa: E731
    want = [run(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[run(x, stream=s) for x, s in zip(xs, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("T, E, H, I, topk", [(1, 40, 128, 384, 8), (3, 24, 640, 1408, 8), (40, 40, 128, 384, 8)])
def test_layers_that_read_what_the_last_one_wrote(T, E, H, I, topk):
    """Layer after layer in place, launched one after the other while the last one ends: the
    same bits as with a wait after every call."""
    lay = layer(E, H, I)
    wr = (torch.randn(E, H, generator=torch.Generator().manual_seed(13)) * 0.1).to(torch.bfloat16).cuda()

    def chain(wait):
        x, seen = synth.activations(T, H, seed=T).cuda(), []
        for k in range(30):
            _, ids, w = nvq.w4a16_moe(x, wr, lay.gate_up, lay.down, I, topk, residual=x, y=x)
            if k % 4 == 1:
                lay(x, ids, w, residual=x, y=x)              # the experts alone, with the same choices
            if wait:
                torch.cuda.synchronize()
            x = (x.float() / x.float().square().mean(1, keepdim=True).sqrt()).to(torch.bfloat16)   # a layer's output grows with the square of x
            seen.append(ids)
        return x, torch.stack(seen)

    want = chain(True)
    assert torch.isfinite(want[0]).all()
    for _ in range(3):
        got = chain(False)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_captured_layer_follows_new_inputs():
    lay = layer(8, 256, 128)
    g = torch.Generator().manual_seed(12)
    wr = (torch.randn(8, 256, generator=g) * 0.1).to(torch.bfloat16).cuda()
    x = synth.activations(6, 256, seed=1).cuda()
    ids, w = torch.empty(6, 2, dtype=torch.int32, device="cuda"), torch.empty(6, 2, device="cuda")
    run = lambda **kw: nvq.w4a16_moe(x, wr, lay.gate_up, lay.down, 128, 2, residual=x, **kw)       # noqa: E731
    run()
    y = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            run(ids=ids, weights=w, y=y)
    for seed in range(2, 6):
        x.copy_(synth.activations(6, 256, seed=seed))
        graph.replay()
        got = y.clone(), ids.clone(), w.clone()
        assert all(torch.equal(p, q) for p, q in zip(got, run()))


def test_decoder_block_tail_in_place_on_one_residual_stream():
    """o_proj added to the stream, then the experts added to it, captured and run over several steps,
    against the oracle applied to the same BF16 stream."""
    T, E, H, I, topk = 5, 8, 256, 128, 2
    lay = layer(E, H, I)
    g = torch.Generator().manual_seed(13)
    wo = (torch.randn(H, 384, generator=g) * 0.05).to(torch.bfloat16)
    wr = (torch.randn(E, H, generator=g) * 0.1).to(torch.bfloat16)
    wr_gpu = wr.cuda()
    c, s = nvq.int4_quantize(wo.cuda())
    packed = nvq.int4_pack_weights(c, s, H, 384)
    u, sb = oracle_int4(wo)
    attn, stream = synth.activations(T, 384, seed=1).cuda(), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    mid = torch.empty_like(stream)
    ids, w = torch.empty(T, topk, dtype=torch.int32, device="cuda"), torch.empty(T, topk, device="cuda")

    def step():
        nvq.nvq_linear_epilogue(attn, None, packed, H, residual=stream, y=mid)
        nvq.w4a16_moe(mid, wr_gpu, lay.gate_up, lay.down, I, topk, residual=mid, ids=ids, weights=w, y=stream)

    stream.zero_()
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    from oracle import epilogue as oepi
    for seed in range(3):
        attn.copy_(synth.activations(T, 384, seed=20 + seed))
        stream.copy_(torch.randn(T, H, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16))
        before = stream.cpu()
        graph.replay()
        want, tol = oepi.apply(bf16_to_f64(attn) @ oint4.dequantize(u, sb).T, residual=bf16_to_f64(before))
        assert (np.abs(bf16_to_f64(mid) - want) <= tol).all()
        _check_route(mid.cpu(), wr, topk, True, ids, w)
        _check(stream, *lay.oracle(mid.cpu(), ids, w, mid.cpu()))


def test_binding_refusals():
    lay = layer(8, 256, 128)
    x = synth.activations(4, 256, seed=1).cuda()
    ids, w = (t.cuda() for t in _choices(4, 8, 2, 1))
    for a in ((x.float(), ids, w), (x.t().contiguous().t(), ids, w), (x, ids.long(), w), (x, ids, w.double()), (x, ids[:3], w),
              (x, ids, w[:, :1]), (x, ids.cpu(), w), (x, ids.t().contiguous().t(), w)):
        with pytest.raises(ValueError):
            lay(*a)
    for kw in (dict(residual=x[:3]), dict(y=x.float()), dict(workspace=torch.empty(1 << 24, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            lay(x, ids, w, **kw)
    with pytest.raises(ValueError):
        nvq.w4a16_moe_experts(x, ids, w, lay.gate_up, lay.down, 9, 128)                 # more experts than packed
    with pytest.raises(nvq.NvqError, match="topk"):
        nvq.moe_route(x, x[:1].contiguous(), 2)
    with pytest.raises(nvq.NvqError, match="overlaps"):
        big = torch.zeros(6, 256, dtype=torch.bfloat16, device="cuda")
        lay(big[:4], ids, w, y=big[1:5])
