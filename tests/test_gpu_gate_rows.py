"""The gate's gradient for more rows than a grid of one wave each may have."""

import pytest
import torch

import block_scaled_precision_gemm_amd as bsmm

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROWS = 2**26 + 5            # 2^32 threads and some


@pytest.fixture(autouse=True)
def _lib(gpu_lib):
    yield


def test_rows_without_columns():
    drow = torch.ones(ROWS, device=DEV)
    e = torch.empty(ROWS, 0, device=DEV)
    junk = torch.full((ROWS,), float("nan"), device=DEV)    # for the next tensor of that size
    del junk
    _, _, got = bsmm.bsmm_swiglu_backward(e, e.to(torch.int8), e.to(torch.uint8), row_scale=drow)
    assert got.shape == (ROWS,) and not got.any()


def test_rows():
    """The last rows, and some before, as a small call has them."""
    F = 32
    h = torch.randn(64, 2 * F, device=DEV).to(torch.bfloat16)
    _, q, s = bsmm.bsmm_swiglu(h, checkpoint=True)
    da, r = torch.randn(64, F, device=DEV).to(torch.bfloat16), torch.rand(64, device=DEV)
    want, _, drow = bsmm.bsmm_swiglu_backward(da, q, s, row_scale=r)

    def big(t):
        v = torch.zeros(ROWS, *t.shape[1:], dtype=t.dtype, device=DEV)
        for i in (0, ROWS // 2, ROWS - 64):
            v[i:i + 64] = t
        return v

    got, none, dr = bsmm.bsmm_swiglu_backward(big(da), big(q), big(s), row_scale=big(r), act=False)
    assert none is None
    for i in (0, ROWS // 2, ROWS - 64):
        assert torch.equal(got[i:i + 64], want) and torch.equal(dr[i:i + 64], drow)
    assert dr.count_nonzero() == 3 * drow.count_nonzero()
    assert not got[64:2**20].any() and not got[-2**20:-64].any()
