"""The int8 quantiser for more rows than one launch may have."""

import pytest
import torch

import block_scaled_precision_gemm_amd as bsmm

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _lib(gpu_lib):
    yield


@pytest.mark.parametrize("M,K", [(2**26, 8), (2**24 + 5, 1032)])
def test_many_rows(M, K):
    """Rows here and there, and the last ones, as a small call has them; the
    others are zeros, of scale 1."""
    part = torch.randn(70, K, device=DEV).to(torch.bfloat16)
    q0, s0 = bsmm.bsmm_quant_int8_rowwise(part)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    places = (0, 2**23 - 35, M // 4 + 3, M - 70)               # none overlaps another
    for i in places:
        x[i:i + 70] = part
    q = torch.full((M, K), 99, dtype=torch.int8, device=DEV)
    s = torch.full((M, 1), -1.0, device=DEV)
    bsmm.bsmm_quant_int8_rowwise(x, q=q, scale=s)
    for i in places:
        assert torch.equal(q[i:i + 70], q0) and torch.equal(s[i:i + 70], s0.view(70, 1))
        s[i:i + 70] = 1.0
        q[i:i + 70] = 0
    assert (s == 1.0).all()
    for m in range(0, M, 2**22):
        assert not q[m:m + 2**22].any()
