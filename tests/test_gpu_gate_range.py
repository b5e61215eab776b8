"""The gate and its gradient over the whole range of the types, the type's
lowest value (a mask) among it.

Limits: relative ones as in test_gpu_ckpt.py.  Besides, sigma(g) is off by
2^-149 at most where it is subnormal, which is only for |g| up to 104; beyond,
it is 0 where it should be below 2^-150.  So silu(g) = g sigma(g) is off by
104 * 2^-149 < 2^-142 at most, its derivative sigma(g) (1 + g sigma(-g)) by
twice that, and products with u, da and a row's scale by as much times those.
An output in bf16 adds the half of its smallest step, 2^-134.
"""

import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsmm
from oracle import expert as X
from test_gpu_ckpt import REL, TDT, dev, host

pytestmark = pytest.mark.gpu

TOP = 127 * 2.0**121                     # the largest value of a checkpoint
GATES = [-TOP, -1e38, -1e30, -1e9, -1000.0, -200.0, -150.0, -120.0, -104.5, -103.0, -100.0, -95.0,
         -92.0, -90.0, -89.0, -88.5, -88.0, -87.5, -87.0, -60.0, -17.0, -1.0, -1e-20, -1e-39, 0.0,
         1e-39, 1e-20, 1.0, 17.0, 87.0, 88.5, 90.0, 104.5, 1000.0, 1e9,
         1e18]                           # times 2^60 in fp32 too


@pytest.fixture(autouse=True)
def _lib(gpu_lib):
    yield


def gates(F, seed, top=4.0):
    """A row for each of GATES, its elements from half of it on; ups of up to
    `top`."""
    rng = np.random.default_rng(seed)
    g = np.array(GATES)[:, None] * rng.uniform(0.5, 1.0, (len(GATES), F))
    g[:, ::5] = np.array(GATES)[:, None]
    u = rng.uniform(0.5, 1.0, g.shape) * top * rng.choice([-1, 1], g.shape)
    return np.concatenate([g, u], 1).astype(np.float32)


def within(got, want, dt, rel, room):
    step = 2.0**-8 * np.abs(want) + 2.0**-134 if dt == "bf16" else 2.0**-150
    off = np.abs(host(got) - want)
    assert (off <= rel + room + step).all(), np.argwhere(off > rel + room + step)[:8]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("top", [4.0, 2.0**60])
def test_gradient(top, weighted, dt):
    rng = np.random.default_rng(5)
    F = 96
    q, s = bsmm.bsmm_quant_int8_mx(dev(gates(F, 1, top), TDT[dt]))
    h = X.restore(host(q), host(s))
    R = len(h)
    da = dev(rng.standard_normal((R, F)) / top, TDT[dt])
    r = rng.uniform(0.5, 1.0, R).astype(np.float32) if weighted else None
    dh, act, drow = bsmm.bsmm_swiglu_backward(da, q, s, row_scale=dev(r) if weighted else None)
    eh, ea, er = X.swiglu_backward(host(da), h, r)
    g, u, d = h[:, :F], h[:, F:], host(da)
    one = np.ones((R, 1)) if r is None else r[:, None].astype(np.float64)
    terms = X.sigmoid(g) * (1 + np.abs(g) * X.sigmoid(-g))
    rel = 2 * REL * np.concatenate([np.abs(one * d * u) * terms, np.abs(eh[:, F:])], 1)
    room = 2.0**-141 * np.concatenate([np.abs(one * d * u), np.abs(one * d)], 1)
    within(dh, eh, dt, rel, room)
    within(act, ea, dt, REL * np.abs(ea), 2.0**-141 * np.abs(one * u))
    if weighted:
        total = np.abs(d * X.swiglu(h)).sum(1)
        within(drow, er, "f32", (REL + F * 2.0**-24) * total, 2.0**-141 * np.abs(d * u).sum(1))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gradient_of_large_ups(dt):
    """da * u leaves fp32 where the slope brings their product back into it."""
    F, rng = 64, np.random.default_rng(6)
    low = [g for g in GATES if g <= -60]
    g = np.repeat(np.array(low)[:, None], F, 1)
    u = np.where(rng.random(g.shape) < 0.5, -1, 1) * 2.0**120
    q, s = bsmm.bsmm_quant_int8_mx(dev(np.concatenate([g, u], 1).astype(np.float32), TDT[dt]))
    h = X.restore(host(q), host(s))
    d = rng.uniform(2.0**11, 2.0**12, u.shape).astype(np.float32)
    da, r = dev(d, TDT[dt]), np.full(len(low), 2.0, np.float32)
    dh, act, drow = bsmm.bsmm_swiglu_backward(da, q, s, row_scale=dev(r))
    eh, ea, er = X.swiglu_backward(host(da), h, r)
    g, u, d = h[:, :F], h[:, F:], 2 * host(da)
    terms = X.sigmoid(g) * (1 + np.abs(g) * X.sigmoid(-g))
    within(dh, eh, dt, 2 * REL * np.concatenate([np.abs(d * u) * terms, np.abs(eh[:, F:])], 1),
           2.0**-141 * np.concatenate([np.abs(d * u), np.abs(d)], 1))
    within(act, ea, dt, REL * np.abs(ea), 2.0**-140 * np.abs(u))
    total = np.abs(host(da) * X.swiglu(h)).sum(1)
    within(drow, er, "f32", (REL + F * 2.0**-24) * total, 2.0**-141 * np.abs(d * u).sum(1))


def test_masked_gate():
    """A gate at the type's lowest value passes nothing on, in either direction."""
    h = torch.full((3, 128), 2.0, device="cuda:0", dtype=torch.bfloat16)
    h[1, :64] = torch.finfo(torch.bfloat16).min
    a, q, s = bsmm.bsmm_swiglu(h, checkpoint=True)
    da, r = torch.ones_like(a), torch.ones(3, device="cuda:0")
    dh, act, drow = bsmm.bsmm_swiglu_backward(da, q, s, row_scale=r)
    assert not a[1].any() and not dh[1].any() and not act[1].any() and drow[1] == 0
    assert a[0].all() and torch.equal(a[0], a[2]) and torch.equal(dh[0], dh[2])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("top", [4.0, 2.0**60])
def test_gate(top, dt):
    """Where e^-g leaves fp32 or its reciprocal is subnormal too."""
    h = dev(gates(96, 2, top), TDT[dt])
    a = bsmm.bsmm_swiglu(h)
    want, u = X.swiglu(host(h)), host(h)[:, 96:]
    within(a, want, dt, REL * np.abs(want), 2.0**-141 * np.abs(u))
    assert torch.equal(a, bsmm.bsmm_swiglu(h, checkpoint=True)[0])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_infinite_gates(dt):
    """silu(inf) is inf, silu(-inf) = -inf * 0 a NaN, as in the formula."""
    h = torch.ones(2, 64, device="cuda:0", dtype=TDT[dt])
    h[0, 3], h[1, 4] = float("inf"), float("-inf")
    a = host(bsmm.bsmm_swiglu(h))
    assert a[0, 3] == np.inf and np.isnan(a[1, 4]) and np.isfinite(a).sum() == 62
