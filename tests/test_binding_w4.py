"""What the binding of the 4-bit weight operations and the router refuses
before it calls the library (no GPU needed)."""

import pytest
import torch

import block_scaled_precision_gemm_amd as bsmm


def t(*shape, dt=torch.bfloat16):
    return torch.zeros(*shape, dtype=dt)


U8, F, I = torch.uint8, torch.float32, torch.int32


@pytest.mark.parametrize("call", [
    lambda: bsmm.bsmm_quant_w4(t(4, 128, dt=torch.float16)),
    lambda: bsmm.bsmm_quant_w4(t(4, 128), group=16),
    lambda: bsmm.bsmm_quant_w4(t(4, 96), group=64),
    lambda: bsmm.bsmm_quant_w4(t(4, 128), scale_dtype="f16"),
    lambda: bsmm.bsmm_w4_mm(t(128), t(8, 64, dt=U8), t(8, 1)),
    lambda: bsmm.bsmm_w4_mm(t(2, 128, dt=torch.float16), t(8, 64, dt=U8), t(8, 1)),
    lambda: bsmm.bsmm_w4_mm(t(2, 128), t(8, 64, dt=torch.int8), t(8, 1)),
    lambda: bsmm.bsmm_w4_mm(t(2, 128), t(8, 32, dt=U8), t(8, 1)),
    lambda: bsmm.bsmm_w4_mm(t(2, 128), t(8, 64, dt=U8), t(7, 1)),
    lambda: bsmm.bsmm_w4_mm(t(2, 128), t(8, 64, dt=U8), t(8, 3)),
    lambda: bsmm.bsmm_w4_mm(t(2, 128), t(8, 64, dt=U8), t(8, 1), t(8, 2, dt=U8)),
    lambda: bsmm.bsmm_w4_mm(t(2, 128), t(8, 64, dt=U8), t(8, 1), t(8, 1)),
    lambda: bsmm.bsmm_w4_mm(t(128, 2).t(), t(8, 64, dt=U8), t(8, 1)),
    lambda: bsmm.bsmm_w4_mm(t(2, 128), t(64, 8, dt=U8).t(), t(8, 1)),
    lambda: bsmm.bsmm_w4_mm(t(2, 128), t(8, 64, dt=U8), t(2, 8).t()),
    lambda: bsmm.bsmm_w4_mm(t(2, 128), t(8, 64, dt=U8), t(8, 1), out=t(2, 9)),
    lambda: bsmm.bsmm_w4_mm(t(2, 128), t(8, 64, dt=U8), t(8, 1), out=t(2, 8, dt=F)),
    lambda: bsmm.bsmm_w4_mm(t(2, 128), t(8, 64, dt=U8), t(8, 1), out_dtype="f16"),
    lambda: bsmm.bsmm_w4_expert_mm(t(2, 128), t(8, 64, dt=U8), t(8, 1), None, t(2, dt=I),
                                   t(3, dt=I)),
    lambda: bsmm.bsmm_w4_expert_mm(t(2, 128), t(2, 8, 64, dt=U8), t(2, 8, 1), None, t(2, dt=F),
                                   t(3, dt=I)),
    lambda: bsmm.bsmm_w4_expert_mm(t(2, 128), t(2, 8, 64, dt=U8), t(2, 8, 1), None, t(2, dt=I),
                                   t(2, dt=I)),
    lambda: bsmm.bsmm_w4_expert_mm(t(2, 128), t(2, 8, 64, dt=U8), t(2, 8, 1), None, t(2, dt=I),
                                   t(3, dt=I), row_scale=t(3, dt=F)),
    lambda: bsmm.bsmm_route_topk(t(4, 8, dt=I), 2),
    lambda: bsmm.bsmm_route_topk(t(8, dt=F), 2),
    lambda: bsmm.bsmm_route_topk(t(4, 8, dt=F), 0),
    lambda: bsmm.bsmm_route_topk(t(4, 8, dt=F), 9),
    lambda: bsmm.bsmm_route_topk(t(8, 4, dt=F).t(), 2),
    lambda: bsmm.bsmm_route_topk(t(4, 8, dt=F), 2, mask=t(4, dt=F)),
    lambda: bsmm.bsmm_route_topk(t(4, 8, dt=F), 2, mask=t(5, dt=U8)),
    lambda: bsmm.bsmm_route_topk_backward(t(4, 8, dt=F), t(4, 2, dt=F), t(4, 2, dt=F),
                                          t(8, dt=I), t(1, dt=I)),
    lambda: bsmm.bsmm_route_topk_backward(t(4, 8, dt=F), t(3, 2, dt=I), t(4, 2, dt=F),
                                          t(8, dt=I), t(1, dt=I)),
    lambda: bsmm.bsmm_route_topk_backward(t(4, 8, dt=F), t(4, 2, dt=I), t(4, 3, dt=F),
                                          t(8, dt=I), t(1, dt=I)),
    lambda: bsmm.bsmm_route_topk_backward(t(4, 8, dt=F), t(4, 2, dt=I), t(4, 2, dt=F),
                                          t(7, dt=I), t(1, dt=I), dloss=t(1, dt=F)),
    lambda: bsmm.bsmm_route_topk_backward(t(4, 8, dt=F), t(4, 2, dt=I), t(4, 2, dt=F),
                                          t(8, dt=I), None, dloss=t(1, dt=F)),
    lambda: bsmm.bsmm_route_topk_backward(t(4, 8, dt=F), t(4, 2, dt=I), t(4, 2, dt=F),
                                          t(8, dt=I), t(1, dt=I), dweight=t(4, 2)),
])
def test_rejects(call):
    with pytest.raises(ValueError):
        call()
