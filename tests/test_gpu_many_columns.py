"""A GEMM of few rows by more columns than a launch of one workgroup per 16 of
them may have (2^32 threads)."""

import pytest
import torch

import block_scaled_precision_gemm_amd as bsmm

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _lib(gpu_lib):
    yield


@pytest.mark.parametrize("M", [1, 17])
def test_int8(M):
    """34 GB of weights: zeros but for three runs of columns."""
    N, K = 2**28 + 64, 128
    g = torch.Generator(device=DEV).manual_seed(M)
    a = torch.randint(-128, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
    part = torch.randint(-128, 128, (70, K), generator=g, device=DEV, dtype=torch.int8)
    b = torch.zeros(N, K, dtype=torch.int8, device=DEV)
    places = (0, N // 2 + 3, N - 70)
    for i in places:
        b[i:i + 70] = part
    out = torch.full((M, N), -7, dtype=torch.int32, device=DEV)
    bsmm.bsmm_int8_rowwise(a, b.t(), out_dtype="i32", out=out)
    want = (a.cpu().long() @ part.cpu().long().t()).to(torch.int32)
    for i in places:
        assert torch.equal(out[:, i:i + 70].cpu(), want)
        out[:, i:i + 70] = 0
    assert not out.any()
