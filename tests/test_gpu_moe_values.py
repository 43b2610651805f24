"""Experts whose h leaves FP32's range: the formula's infinities, not NaN, and only where they belong.

Every gate, up and down row holds one value, so that no term is 0 * inf and all terms of a sum have
one sign: the formula in any arithmetic that overflows gives the signed infinity.
"""
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


def _pack(w):
    return nvq.int4_pack_weights(*nvq.int4_quantize(w.cuda()), *w.shape)


# few units and many (eight and sixteen warps per CTA), h staged in shared memory or not, one and two MMA tiles per segment
@pytest.mark.parametrize("T, E, H, I, topk", [(1, 1, 128, 128, 1), (3, 8, 256, 128, 2), (9, 1, 128, 384, 1), (32, 4, 256, 256, 2),
                                              (2, 8, 4096, 512, 4), (32, 8, 2048, 768, 2), (40, 2, 256, 128, 2)])
@pytest.mark.parametrize("value", [1e18, 2e30, float("inf")])
def test_an_infinite_h_gives_an_infinite_y(T, E, H, I, topk, value):
    ones = torch.ones(E * I, H, dtype=torch.bfloat16)
    gate_up = _pack(torch.cat([nvq.interleave_gate_up(ones[:I], ones[:I], block=16)] * E))
    sign = torch.where(torch.arange(H) % 3 == 0, -1.0, 1.0).to(torch.bfloat16)
    down = _pack(sign.unsqueeze(1).expand(H, I).repeat(E, 1).contiguous())
    ids = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:topk] for t in range(T)]).int().cuda()
    w = torch.full((T, topk), 0.5).cuda()
    x = torch.full((T, H), 0.25, dtype=torch.bfloat16)
    res = torch.randn(T, H, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16).cuda()
    call = lambda x: nvq.w4a16_moe_experts(x.cuda(), ids, w, gate_up, down, E, I, residual=res)    # noqa: E731
    plain = call(x)
    assert torch.isfinite(plain).all()
    big = T // 2
    x[big] = value
    y = call(x)
    assert torch.equal(y[big].float().cpu(), float("inf") * sign.float())
    rest = [t for t in range(T) if t != big]
    assert torch.equal(y[rest], plain[rest])
