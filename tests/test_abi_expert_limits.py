"""Sizes of the experts' products next to 2^31, where their kernels' 32-bit
counts of elements, a tile past the last one, would wrap: refused, before any
HIP call and so without a GPU (see test_abi_expert.py)."""

import pytest

import block_scaled_precision_gemm_amd as bsmm
from test_abi_expert import BF16, F32, UNSUP, mm, wgrad

TOP = 2**31 - 1024


@pytest.mark.parametrize("n", [TOP, TOP + 1, 2**31 - 64, 2**31 - 1, 2**31])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_refused(n, dt):
    assert mm(dt=dt, E=1, K=n, ldx=2**31, w_sn=2**31, w_se=2**36) == UNSUP
    assert mm(dt=dt, E=1, K=n, ldx=2**31, w_sn=1, w_sk=32, w_se=2**36) == UNSUP
    assert mm(dt=dt, E=1, R=1, S=1, per=1, N=n, ldo=2**31) == UNSUP
    assert mm(dt=dt, E=1, R=1, S=1, per=1, N=n, ldo=2**31, w_sn=1, w_sk=2**31) == UNSUP
    assert wgrad(dt=dt, E=1, N=n, ldy=2**31, w_se=2**62) == UNSUP
    assert wgrad(dt=dt, E=1, K=n, ldx=2**31, ldw=2**31, w_se=2**62) == UNSUP
    code = "bf16" if dt == BF16 else "f32"
    for size in ((n, 64, 64), (64, n, 64), (64, 64, n)):
        assert bsmm.bsmm_expert_mm_plan_name(code, False, 1, *size) is None
        assert bsmm.bsmm_expert_mm_workspace_bytes(code, False, 1, *size) == 0
        assert bsmm.bsmm_expert_wgrad_plan_name(code, False, 1, 64, *size) is None
        assert bsmm.bsmm_expert_wgrad_workspace_bytes(code, False, 1, 64, *size) == 0


@pytest.mark.parametrize("kw", [
    # few rows of many experts by very many columns
    dict(E=1024, R=1024, S=1024, per=1, N=2**24, K=1, ldx=1, w_sn=1, w_se=0, ldo=2**24),
    dict(E=1024, R=1024, S=1024, per=1, N=2**24, K=8, ldx=9, w_sn=8, w_se=0, ldo=2**24),
    # very many rows
    dict(dt=F32, E=1, R=2**30, S=2**30, per=1, N=16, K=8, ldx=8, w_sn=8, w_se=0, ldo=16),
])
def test_grids_of_more_threads_than_32_bits_count(kw):
    """Such a launch runs as many as the low 32 bits say, and reports nothing."""
    assert mm(**kw) == UNSUP


def test_gradient_grids_of_more_threads_than_32_bits_count():
    assert wgrad(dt=F32, E=1024, N=2**14, K=2**13, ldy=2**14, ldx=2**13, ldw=2**13,
                 w_se=2**27) == UNSUP
