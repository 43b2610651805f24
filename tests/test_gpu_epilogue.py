"""The products with bias, activation and residual against the float64 oracle.

Tolerance: oracle.epilogue.apply (its docstring derives it).  Inputs are seeded.
"""
import numpy as np
import pytest
import torch

import phase_disaggregated_quantized_b200 as nvq
from phase_disaggregated_quantized_b200 import synth
from oracle import epilogue as oepi
from oracle import int4 as oint4
from oracle import nvfp4 as onv

from helpers import bf16_bits, bf16_to_f64, oracle_int4, oracle_nvfp4

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


def _draw(M, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = synth.activations(M, K, seed=seed)
    w = (torch.randn(N, K, generator=g) * 0.02).to(torch.bfloat16)
    bias = torch.randn(N, generator=g).to(torch.bfloat16)
    res = torch.randn(M, N, generator=g).to(torch.bfloat16)
    return x, w, bias, res


class Int4:
    """W4A16: quantized and packed once; v of the oracle on demand."""
    step_n, step_k = 32, 128

    def __init__(self, x, w):
        self.x, self.N = x.cuda(), w.shape[0]
        c, s = nvq.int4_quantize(w.cuda())
        self.w = nvq.int4_pack_weights(c, s, *w.shape)
        u, sb = oracle_int4(w)
        self.v = bf16_to_f64(x) @ oint4.dequantize(u, sb).T

    def __call__(self, **kw):
        return nvq.w4a16_gemm_epilogue(self.x, *self.w, self.N, **kw)

    def bare(self):
        return nvq.w4a16_gemm(self.x, *self.w, self.N)


class Nvfp4:
    step_n, step_k = 8, 64

    def __init__(self, x, w):
        self.M, self.K, self.N = *x.shape, w.shape[0]
        self.x, self.w = nvq.nvfp4_quantize(x.cuda()), nvq.nvfp4_quantize(w.cuda())
        (xc, xs, xt), (wc, ws, wt) = onv.quantize(bf16_to_f64(x)), onv.quantize(bf16_to_f64(w))
        self.v = onv.dequantize(xc, xs, xt) @ onv.dequantize(wc, ws, wt).T

    def __call__(self, **kw):
        return nvq.nvfp4_gemm_w4a4_epilogue(self.x, self.w, self.M, self.N, self.K, **kw)

    def bare(self):
        return nvq.nvfp4_gemm_w4a4(self.x, self.w, self.M, self.N, self.K)


def _check(y, v, bias, act, res):
    f = lambda t: None if t is None else bf16_to_f64(t)                                  # noqa: E731
    want, tol = oepi.apply(v, f(bias), act, f(res))
    off = np.abs(bf16_to_f64(y) - want)
    assert (off <= tol).all(), f"worst {np.max(off / tol):.3f} of the tolerance"


def _cu(t):
    return None if t is None else t.cuda()


INT4_SHAPES = [(1, 32, 128), (1, 4096, 256), (7, 96, 384), (8, 2080, 1152), (9, 64, 128), (16, 352, 4096),
               (17, 32, 256), (32, 1056, 384), (33, 96, 128), (70, 64, 640),
               # more than 8 rows: k-groups cut over 8, 4 or 2 CTAs, several rounds of tiles, tiles of one group,
               # whole tiles and then shared ones, several rounds of shared ones
               (12, 64, 8192), (20, 96, 1152), (13, 2080, 2048), (25, 8224, 1024), (16, 18976, 128), (24, 19104, 640),
               (320, 1920, 2048), (320, 1920, 6144), (320, 1024, 16384), (896, 1024, 16384)]
NVFP4_SHAPES = [(1, 8, 64), (5, 264, 128), (31, 72, 192), (128, 256, 256), (129, 520, 1088), (300, 1000, 320),
                (1030, 2312, 64),
                # few tiles, whose k-stages 8, 4 or 2 CTAs split
                (5, 264, 2112), (1, 8, 4096), (129, 1032, 2048), (300, 2312, 832), (257, 3600, 768), (40, 16, 704)]
SHAPES = [(Int4, s) for s in INT4_SHAPES] + [(Nvfp4, s) for s in NVFP4_SHAPES]


@pytest.mark.parametrize("form, shape", SHAPES, ids=lambda p: p.__name__ if isinstance(p, type) else "x".join(map(str, p)))
def test_every_epilogue_matches_the_oracle(form, shape):
    M, N, K = shape
    x, w, bias, res = _draw(M, N, K, seed=M + N + K)
    op = form(x, w)
    for act in oepi.ACTIVATIONS:
        for b in (None, bias):
            for r in (None, res):
                _check(op(bias=_cu(b), activation=act, residual=_cu(r)), op.v, b, act, r)
    nvq.check_device_error()


@pytest.mark.parametrize("form", [Int4, Nvfp4])
def test_empty_epilogue_is_the_bare_product_bit_for_bit(form):
    x, w, _, _ = _draw(6 if form is Int4 else 24, 160, 512, seed=3)
    op = form(x, w)
    assert torch.equal(op(), op.bare())


@pytest.mark.parametrize("form, M", [(Int4, 5), (Int4, 40), (Nvfp4, 40), (Nvfp4, 260)])
def test_residual_stream_updated_in_place(form, M):
    x, w, bias, res = _draw(M, 288, 384, seed=M)
    op = form(x, w)
    stream = res.cuda()
    apart = op(bias=bias.cuda(), residual=res.cuda(), activation="silu")
    got = op(bias=bias.cuda(), residual=stream, activation="silu", y=stream)
    assert got is stream and torch.equal(stream, apart)


@pytest.mark.parametrize("form, M", [(Int4, 1), (Int4, 3), (Int4, 21), (Nvfp4, 3), (Nvfp4, 140)])
def test_strided_rows_and_what_lies_between_them(form, M):
    """y and residual as column ranges of wider buffers, once two ranges of the same buffer."""
    N = 96
    x, w, bias, res = _draw(M, N, 256, seed=M + 1)
    op = form(x, w)
    want = op(bias=bias.cuda(), residual=res.cuda())
    wide = torch.full((M, 3 * N + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    before = wide.clone()
    wide[:, 2 * N:3 * N] = res.cuda()
    before[:, 2 * N:3 * N] = res.cuda()
    op(bias=bias.cuda(), residual=wide[:, 2 * N:3 * N], y=wide[:, 8:8 + N])
    assert torch.equal(wide[:, 8:8 + N], want)
    wide[:, 8:8 + N] = before[:, 8:8 + N]
    assert torch.equal(wide, before)                       # nothing else was written
    # each on its own stride
    ybuf = torch.zeros(M + 1, N + 16, dtype=torch.bfloat16, device="cuda")
    rbuf = torch.zeros(M, N + 40, dtype=torch.bfloat16, device="cuda")
    rbuf[:, 16:16 + N] = res.cuda()
    op(bias=bias.cuda(), residual=rbuf[:, 16:16 + N], y=ybuf[:M, :N])
    assert torch.equal(ybuf[:M, :N], want)
    assert not ybuf[M].any() and not ybuf[:, N:].any()     # the row behind the last and the gap


@pytest.mark.parametrize("form", [Int4, Nvfp4])
def test_values_that_are_not_finite_stay_where_they_are(form):
    M, N = 20, 96
    x, w, bias, res = _draw(M, N, 256, seed=9)
    res[3, 5], res[7, 95], res[19, 0] = float("nan"), float("inf"), float("-inf")
    bias[11] = float("inf")
    op = form(x, w)
    y = op(bias=bias.cuda(), activation="relu", residual=res.cuda()).float().cpu()
    assert torch.isnan(y[3, 5]) and y[7, 95] == float("inf") and y[19, 0] == float("-inf")
    assert (y[:, 11] == float("inf")).all()
    y[3, 5] = y[7, 95] = y[19, 0] = 0
    y[:, 11] = 0
    assert torch.isfinite(y).all()
    bias[11] = float("nan")
    for act in oepi.ACTIVATIONS:
        y = op(bias=bias.cuda(), activation=act).float().cpu()
        assert torch.isnan(y[:, 11]).all() and torch.isfinite(y[:, :11]).all() and torch.isfinite(y[:, 12:]).all()


@pytest.mark.parametrize("M, N, K", [(9, 96, 256), (16, 160, 1152), (17, 96, 256), (32, 288, 2048), (45, 64, 640)])
def test_int4_sums_of_integers_are_exact(M, N, K):
    """Integer x, every code, power-of-two scales: the FP32 sums hold the result exactly, y is its one rounding."""
    g = torch.Generator().manual_seed(M)
    x = torch.randint(-8, 9, (M, K), generator=g).to(torch.bfloat16)
    u = torch.randint(0, 16, (N, K), generator=g, dtype=torch.uint8)
    s = torch.exp2(torch.randint(-2, 3, (N, K // 128), generator=g).float()).to(torch.bfloat16)
    packed = nvq.int4_pack_weights((u[:, 0::2] | (u[:, 1::2] << 4)).cuda(), s.cuda(), N, K)
    y = nvq.w4a16_gemm_epilogue(x.cuda(), *packed, N)
    w = (u.double() - 8) * s.double().repeat_interleave(128, 1)
    want = x.double() @ w.T                                 # |sums| < 2^21, multiples of 2^-2
    assert torch.equal(y.cpu(), want.float().to(torch.bfloat16))


@pytest.mark.parametrize("M", [9, 16, 19, 31, 50])
def test_rows_do_not_see_one_another(M):
    """A row of NaN, and NaN behind the last row, change nothing but that row."""
    x, w, bias, _ = _draw(M, 160, 1024, seed=M)
    op = Int4(x, w)
    want = op(bias=bias.cuda())
    wide = torch.full((M + 70, 1024), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:M] = op.x
    wide[3] = float("nan")
    op.x = wide[:M]
    y = op(bias=bias.cuda())
    assert torch.isnan(y[3]).all()
    y[3] = want[3]
    assert torch.equal(y, want)


@pytest.mark.parametrize("act", oepi.ACTIVATIONS)
def test_activations_over_their_range(act):
    """x of all zeros: the result is act(bias), over large, tiny and border arguments."""
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e-4, -1e-4, 0.5, -0.5, 1.0, -1.0, 3.0, -3.0, 6.0, -6.0, 20.0, -20.0,
                      80.0, -80.0, 88.5, -88.5, 100.0, -100.0, 1e10, -1e10, 3e38, -3e38] + [0.0] * 6).to(torch.bfloat16)
    x, w, _, _ = _draw(2, 32, 128, seed=4)
    for op in (Int4(torch.zeros_like(x), w), Nvfp4(torch.zeros_like(x), w)):
        y = bf16_to_f64(op(bias=z.cuda(), activation=act))
        want = oepi.activation(bf16_to_f64(z), act)
        # half a BF16 step, the fast exponential's 1e-5, FP32 sums next to 1, and results below 1e-30 may be 0
        tol = (2.0 ** -8 + 1e-5) * np.abs(want) + 2.0 ** -22 * np.abs(bf16_to_f64(z)) * (act == "gelu") + 1e-30
        assert (np.abs(y - want) <= tol).all()


def test_repeated_and_concurrent_calls_agree():
    """Two products at once on two streams, and each again: the same bits."""
    x, w, bias, res = _draw(16, 1056, 1152, seed=5)
    a, b = Int4(x, w), Nvfp4(x, w)
    ra, rb = a(bias=bias.cuda(), residual=res.cuda()), b(bias=bias.cuda(), residual=res.cuda())
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    bc, rc = bias.cuda(), res.cuda()
    torch.cuda.synchronize()
    ys = []
    for _ in range(10):
        ys.append((a(bias=bc, residual=rc, stream=s1), b(bias=bc, residual=rc, stream=s2)))
    torch.cuda.synchronize()
    for p, q in ys:
        assert torch.equal(p, ra) and torch.equal(q, rb)


@pytest.mark.parametrize("M", [4, 20, 50])
def test_captured_and_replayed_on_new_inputs(M):
    x, w, bias, res = _draw(M, 256, 256, seed=6)
    op = Int4(x, w)
    stream = res.cuda()
    op(bias=bias.cuda(), residual=stream.clone(), activation="gelu")
    bc = bias.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        op(bias=bc, residual=stream, y=stream, activation="gelu")
        op(bias=bc, residual=stream, y=stream, activation="gelu")     # reads what the first wrote
    for seed in (7, 8):
        x2, _, _, res2 = _draw(M, 256, 256, seed=seed)
        op.x.copy_(x2)
        stream.copy_(res2)
        g.replay()
        want = op(bias=bc, residual=op(bias=bc, residual=res2.cuda(), activation="gelu"), activation="gelu")
        assert torch.equal(stream, want)


@pytest.mark.parametrize("M", [1, 8, 12, 20, 40])
@pytest.mark.parametrize("form", ["w4a16", "w4a4", "both"])
def test_calls_that_read_what_the_last_one_wrote(form, M):
    """Forty calls on two buffers, each reading one and updating the other, launched one after
    the other while the last one ends: the same bits as with a wait after every call."""
    N = 512
    _, w, bias, res = _draw(M, N, N, seed=M)
    i4 = nvq.int4_pack_weights(*nvq.int4_quantize(w.cuda()), N, N)
    f4, bc = nvq.nvfp4_quantize(w.cuda()), (0.1 * bias).cuda()

    def chain(wait):
        a, b = res.cuda(), (0.5 * res).cuda()
        for k in range(40):
            if form == "w4a16" or (form == "both" and k % 3 != 2):
                nvq.w4a16_gemm_epilogue(a, *i4, N, bias=bc, activation="silu", residual=b, y=b)
            else:
                nvq.nvfp4_gemm_w4a4_epilogue(nvq.nvfp4_quantize(a), f4, M, N, N, bias=bc, activation="silu", residual=b, y=b)
            if wait:
                torch.cuda.synchronize()
            b = 0.75 * b if k % 5 == 4 else b                # a kernel of another kind in between
            a, b = b, a
        return a, b

    want = chain(True)
    for _ in range(3):
        got = chain(False)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.isfinite(want[0]).all()


@pytest.mark.parametrize("M", [1, 16, 17, 200])
def test_phase_dispatch_takes_the_epilogue_along(M):
    x, w, bias, res = _draw(M, 160, 256, seed=M)
    i4, f4 = Int4(x, w), Nvfp4(x, w)
    kw = dict(bias=bias.cuda(), activation="gelu_tanh", residual=res.cuda())
    got = nvq.nvq_linear_epilogue(x.cuda(), f4.w, i4.w, 160, **kw)
    assert torch.equal(got, i4(**kw) if M <= nvq.default_crossover_m() else f4(**kw))
    assert torch.equal(nvq.nvq_linear_epilogue(x.cuda(), f4.w, None, 160, crossover_m=0, **kw), f4(**kw))
    assert torch.equal(nvq.nvq_linear_epilogue(x.cuda(), None, i4.w, 160, crossover_m=10 ** 6, **kw), i4(**kw))
    if not 8 < M <= nvq.default_crossover_m():              # there the INT4 product has sums in an order of its own
        assert torch.equal(nvq.nvq_linear_epilogue(x.cuda(), f4.w, i4.w, 160), nvq.nvq_linear(x.cuda(), f4.w, i4.w, 160))


def test_binding_refusals():
    x, w, bias, res = _draw(4, 64, 128, seed=1)
    op = Int4(x, w)
    for kw in (dict(bias=bias), dict(bias=bias.cuda()[:32]), dict(bias=bias.cuda().float()),
               dict(residual=res.cuda()[:3]), dict(residual=res.cuda().t().contiguous().t()), dict(activation="tanh"),
               dict(y=res.cuda().float())):
        with pytest.raises(ValueError):
            op(**kw)
    y = torch.empty(4, 72, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(nvq.NvqError, match="not a multiple of 8"):
        op(y=torch.empty(4, 70, dtype=torch.bfloat16, device="cuda")[:, :64])
    with pytest.raises(nvq.NvqError, match="overlaps"):
        op(y=y[:, :64], residual=y[:, 8:])
    with pytest.raises(ValueError):
        nvq.w4a16_gemm_epilogue(op.x, op.w[0][:100], op.w[1], 64)
    with pytest.raises(ValueError):
        nvq.w4a16_gemm_epilogue(op.x.t(), *op.w, 64)
