"""What the compiled binding refuses by the arguments' form alone, before it looks at a device (no GPU)."""
import pytest
import torch

import phase_disaggregated_quantized_b200 as nvq
from phase_disaggregated_quantized_b200 import build_lib


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_lib.build()


def _bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def products(M, N, K):
    """The three calls with an epilogue on host tensors, which each refuses in the end for being there."""
    x, u8, t = _bf16(M, K), torch.zeros(8, dtype=torch.uint8), torch.zeros(1)
    yield lambda **kw: nvq.nvfp4_gemm_w4a4_epilogue((u8, u8, t), (u8, u8, t), M, N, K, **kw)
    yield lambda **kw: nvq.w4a16_gemm_epilogue(x, u8, u8, N, **kw)
    yield lambda **kw: nvq.nvq_linear_epilogue(x, None, (u8, u8), N, **kw)


@pytest.mark.parametrize("name", ["residual", "y"])
def test_rows_that_share_memory_are_refused(name):
    """Strides of 0 (broadcast) and of less than a row; (0, 1) is what expand gives."""
    N = 32
    assert _bf16(1, N).expand(4, N).stride() == (0, 1)
    for shared in (_bf16(1, N).expand(4, N), _bf16(N).expand(4, N), _bf16(4 * N).as_strided((4, N), (N - 8, 1)),
                   _bf16(4 * N).as_strided((4, N), (8, 1)), _bf16(1, 1).expand(4, N)):
        for call in products(4, N, 128):
            with pytest.raises(ValueError, match="row stride of at least 32"):
                call(**{name: shared})
    for apart in (_bf16(4, N), _bf16(4, 3 * N)[:, 8:8 + N], _bf16(8, N)[::2]):
        for call in products(4, N, 128):
            with pytest.raises(ValueError, match="CUDA"):
                call(**{name: apart})
    for call in products(1, N, 128):                         # one row has no row stride
        with pytest.raises(ValueError, match="CUDA"):
            call(**{name: _bf16(1, 1).expand(1, N)})


def test_experts_take_no_missing_choices():
    """ids and weights are inputs of the experts: nothing stands in for them (moe_route makes them where they are outputs)."""
    x, u8 = _bf16(2, 128), torch.zeros(8, dtype=torch.uint8)
    ids, weights = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, 1)
    call = lambda i, w: nvq.w4a16_moe_experts(x, i, w, (u8, u8), (u8, u8), 2, 128)             # noqa: E731
    with pytest.raises(ValueError, match="weights must be a tensor"):
        call(ids, None)
    with pytest.raises(ValueError, match="ids must be a tensor"):
        call(None, weights)
    with pytest.raises(ValueError, match="CUDA"):
        call(ids, weights)


def test_renormalize_without_a_truth_value_raises_its_own_error():
    class Neither:
        def __bool__(self):
            raise KeyError("neither")

    x, u8 = _bf16(2, 128), torch.zeros(8, dtype=torch.uint8)
    for flag, error in ((Neither(), KeyError), (torch.ones(2), RuntimeError)):
        with pytest.raises(error):
            nvq.moe_route(x, x, 1, renormalize=flag)
        with pytest.raises(error):
            nvq.w4a16_moe(x, x, (u8, u8), (u8, u8), 128, 1, renormalize=flag)
    with pytest.raises(ValueError, match="CUDA"):
        nvq.moe_route(x, x, 1, renormalize=torch.ones(1))
