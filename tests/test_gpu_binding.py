"""The compiled binding on the GPU: arguments it must refuse before anything is launched, and how it calls."""
import pytest
import torch

import phase_disaggregated_quantized_b200 as nvq

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


def products(M, N, K, seed=0):
    """The calls with an epilogue, by both paths of the dispatch."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16).cuda()
    w = torch.randn(N, K, generator=g).to(torch.bfloat16).cuda()
    i4, f4, xq = nvq.int4_pack_weights(*nvq.int4_quantize(w), N, K), nvq.nvfp4_quantize(w), nvq.nvfp4_quantize(x)
    return [lambda **kw: nvq.nvfp4_gemm_w4a4_epilogue(xq, f4, M, N, K, **kw),
            lambda **kw: nvq.w4a16_gemm_epilogue(x, *i4, N, **kw),
            lambda **kw: nvq.nvq_linear_epilogue(x, f4, i4, N, crossover_m=10 ** 6, **kw),
            lambda **kw: nvq.nvq_linear_epilogue(x, f4, i4, N, crossover_m=0, **kw)]


@pytest.mark.parametrize("M", [2, 4, 9, 40, 200])
def test_broadcast_rows_are_refused_and_their_copy_is_not(M):
    N = 64
    row = torch.randn(1, N, generator=torch.Generator().manual_seed(M)).to(torch.bfloat16).cuda()
    before = row.clone()
    for call in products(M, N, 128):
        for kw in (dict(residual=row.expand(M, N)), dict(y=row.expand(M, N)),
                   dict(residual=row.expand(M, N), y=torch.empty(M, N, dtype=torch.bfloat16, device="cuda"))):
            with pytest.raises(ValueError, match="row stride of at least 64"):
                call(**kw)
        # the sum with its copy is the sum with the row as a bias: both are added in FP32, to a product of one rounding
        assert torch.equal(call(residual=row.expand(M, N).contiguous()), call(bias=row[0]))
    assert torch.equal(row, before)


def test_one_row_may_be_broadcast():
    """A single row has no row stride: whatever the view says of it, N elements are there."""
    N = 64
    for call in products(1, N, 128):
        wide = torch.randn(N, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
        assert torch.equal(call(residual=wide.expand(1, N)), call(bias=wide))


def test_experts_take_no_missing_choices():
    E, H, I = 2, 128, 128
    pack = lambda r, c: nvq.int4_pack_weights(*nvq.int4_quantize(torch.ones(r, c, dtype=torch.bfloat16).cuda()), r, c)   # noqa: E731
    gate_up, down = pack(E * 2 * I, H), pack(E * H, I)
    x, ids = torch.ones(3, H, dtype=torch.bfloat16).cuda(), torch.zeros(3, 1, dtype=torch.int32).cuda()
    y = torch.full((3, H), 7.0, dtype=torch.bfloat16).cuda()
    with pytest.raises(ValueError, match="weights must be a tensor"):
        nvq.w4a16_moe_experts(x, ids, None, gate_up, down, E, I, y=y)
    with pytest.raises(ValueError, match="ids must be a tensor"):
        nvq.w4a16_moe_experts(x, None, torch.ones(3, 1).cuda(), gate_up, down, E, I, y=y)
    assert (y == 7).all()


def test_renormalize_without_a_truth_value_launches_nothing():
    x = torch.ones(3, 128, dtype=torch.bfloat16).cuda()
    ids, weights = torch.full((3, 1), 7, dtype=torch.int32).cuda(), torch.full((3, 1), 7.0).cuda()
    with pytest.raises(RuntimeError, match="(?i)bool"):
        nvq.moe_route(x, x, 1, renormalize=torch.ones(2), ids=ids, weights=weights)
    torch.cuda.synchronize()
    assert (ids == 7).all() and (weights == 7).all()


def test_other_threads_run_while_a_call_waits(tmp_path):
    """A call waits on the host when the launch queue is full.  Here the entry points are a C function that
    sleeps 0.3 s and refuses, bound into a copy of the module of its own; another thread counts meanwhile."""
    import ctypes
    import importlib.util
    import shutil
    import subprocess
    import threading
    import time
    src = tmp_path / "slow.c"
    src.write_text("#include <unistd.h>\nint slow(void) { usleep(300000); return 1; }\nunsigned long none(void) { return 0; }\n")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(tmp_path / "slow.so"), str(src)], check=True)
    L = ctypes.CDLL(str(tmp_path / "slow.so"))
    shutil.copy(nvq.BINDING_PATH, tmp_path / "_binding.so")
    spec = importlib.util.spec_from_file_location("slow._binding", tmp_path / "_binding.so")
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    at = lambda f: ctypes.cast(f, ctypes.c_void_p).value                                       # noqa: E731
    m.bind(at(L.slow), at(L.slow), at(L.slow), at(L.none), at(L.slow), at(L.none), at(L.slow), at(L.slow))
    u8 = torch.zeros(1 << 16, dtype=torch.uint8).cuda()
    x, t, ids, w = torch.zeros(2, 128, dtype=torch.bfloat16).cuda(), torch.zeros(1).cuda(), torch.zeros(2, 1, dtype=torch.int32).cuda(), torch.zeros(2, 1).cuda()
    q4, p4 = (u8, u8, t), (u8, u8)
    calls = [lambda: m.nvfp4_gemm_w4a4_epilogue(q4, q4, 2, 64, 128, None, 0, None, None),
             lambda: m.w4a16_gemm_epilogue(x, p4, 64, None, 0, None, None),
             lambda: m.nvq_linear_epilogue(x, q4, p4, 64, None, 0, None, -1, None, None),
             lambda: m.moe_route(x, x, 1, True, None, None),
             lambda: m.w4a16_moe_experts(x, ids, w, p4, p4, 1, 128, None, None, None),
             lambda: m.w4a16_moe(x, x[:1], p4, p4, 128, 1, True, None, None, None, None, None)]
    ticks, stop = [], threading.Event()

    def count():
        while not stop.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.005)

    thread = threading.Thread(target=count)
    thread.start()
    try:
        for call in calls:
            begin = time.perf_counter()
            assert call() == 1
            end = time.perf_counter()
            assert end - begin >= 0.29
            within = [s for s in ticks if begin + 0.05 < s < end - 0.05]
            assert len(within) >= 5                          # 40 with nothing else to do
    finally:
        stop.set()
        thread.join()
