"""8-bit checkpoints and the gate on the GPU.

Codes, bytes and values bit for bit.  The gate in fp32: e^-g has the
instruction's 2^-23 and one rounding each of the corrected exponent and the
correction (2^-24 each), the sum 1 + e^-g one, its reciprocal 2^-23, and up to
four products one each: at most 2^-23 * (1 + 1 + 1/2 + 1 + 2) < 6 * 2^-23 of
the result.  The gradient's slope s (1 + g (1 - s)) has two terms of either
sign, the second with e^-g s for 1 - s: 2 for e^-g, 4 for s and for g s 1/2
more, and two more roundings, below 12 * 2^-23 of the terms' sizes.  A sum of n
terms adds n 2^-24 of their sizes.  An output rounded to bf16 adds 2^-8.
Numbers below 2^-126 may be flushed, before they meet factors below 2^16.
"""

import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsmm
from oracle import expert as X

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TDT = {"bf16": torch.bfloat16, "f32": torch.float32}
REL = 6 * 2.0**-23


@pytest.fixture(autouse=True)
def _lib(gpu_lib):
    yield


def dev(a, dt=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dt is None else t.to(dt)


def host(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def close(got, want, dt, size=None):
    limit = (REL * np.abs(want) if size is None else 12 * 2.0**-23 * size) + 2.0**-110
    limit += 2.0**-8 * np.abs(want) if dt == "bf16" else 0.0
    assert (np.abs(host(got) - want) <= limit).all()


def activations(R, K, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((R, K)) * np.exp2(rng.integers(-20, 20, (R, 1)))
    x[:, ::37] *= 16
    x[rng.random((R, K)) < 0.05] = 0.0
    x[0] = 0.0
    if R > 6:
        x[1] = np.exp2(rng.integers(-149, -120, K).astype(np.float64))   # subnormals and near
        x[2] = np.exp2(127.0) * rng.standard_normal(K).clip(-1.9, 1.9)
        x[3] = (np.arange(K) % 64 + 0.5) / 64                            # ties
        x[4] = 1.999                                                     # beyond code 127
        x[5] = -x[6]
    return x.astype(np.float32)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("R,K", [(1, 32), (7, 96), (33, 1024), (9, 4128), (1000, 64)])
def test_codes_exact(R, K, dt):
    x = dev(activations(R, K, R + K), TDT[dt])
    q, s, v = bsmm.bsmm_quant_int8_mx(x, values=True)
    eq, es, ev = X.quantise(host(x))
    assert q.dtype == torch.int8 and s.dtype == torch.uint8 and v.dtype == x.dtype
    assert np.array_equal(host(s), es) and np.array_equal(host(q), eq)
    assert np.array_equal(host(v), ev)
    q2, s2 = bsmm.bsmm_quant_int8_mx(x)
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_special_blocks(dt):
    x = dev(activations(8, 128, 1), TDT[dt])
    x[3, 40], x[5, 0], x[6, 127] = float("inf"), float("nan"), float("-inf")
    q, s, v = bsmm.bsmm_quant_int8_mx(x, values=True)
    eq, es, ev = X.quantise(host(x))
    assert np.array_equal(host(s), es) and np.array_equal(host(q), eq)
    assert np.array_equal(host(v), ev, equal_nan=True)
    assert (es == 255).sum() == 3


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_of_a_larger_tensor(dt):
    x = dev(activations(6, 256, 2), TDT[dt])
    part = x[:, 64:192]
    q, s = bsmm.bsmm_quant_int8_mx(part)
    eq, es, _ = X.quantise(host(part))
    assert np.array_equal(host(s), es) and np.array_equal(host(q), eq)
    q, s = bsmm.bsmm_quant_int8_mx(x.view(2, 3, 256))
    eq, es, _ = X.quantise(host(x))
    assert np.array_equal(host(q).reshape(6, 256), eq) and s.shape == (2, 3, 8)
    with pytest.raises(bsmm.BsmmError, match="ALIGN"):
        bsmm.bsmm_quant_int8_mx(x[:, 1:65])


GATES = [(1, 32), (8, 2048), (7, 96), (33, 160), (257, 64), (5, 4128)]


def gate_input(R, F, dt, seed):
    rng = np.random.default_rng(seed)
    h = rng.standard_normal((R, 2 * F)) * 4
    h[:, 5] = np.linspace(-120, 120, R)           # to where e^-g leaves fp32
    h[:, 9] = 0.0
    return dev(h, TDT[dt])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("R,F", GATES)
def test_gate(R, F, dt):
    h = gate_input(R, F, dt, R + F)
    a = bsmm.bsmm_swiglu(h)
    assert a.dtype == h.dtype
    close(a, X.swiglu(host(h)), dt)
    b, q, s = bsmm.bsmm_swiglu(h, checkpoint=True)
    eq, es, _ = X.quantise(host(h))
    assert torch.equal(a, b) and np.array_equal(host(q), eq) and np.array_equal(host(s), es)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("R,F", GATES)
def test_gate_gradient(R, F, weighted, dt):
    rng = np.random.default_rng(R * F)
    q, s = bsmm.bsmm_quant_int8_mx(gate_input(R, F, dt, R))
    h = X.restore(host(q), host(s))
    da = dev(rng.standard_normal((R, F)) * 1e-3, TDT[dt])
    r = rng.random(R).astype(np.float32) if weighted else None
    if weighted:
        r[0] = 0.0
    dh, act, drow = bsmm.bsmm_swiglu_backward(da, q, s, row_scale=dev(r) if weighted else None)
    eh, ea, er = X.swiglu_backward(host(da), h, r)
    g, u = h[:, :F], h[:, F:]
    one = 1.0 if r is None else r[:, None]
    terms = X.sigmoid(g) * (1 + np.abs(g) * X.sigmoid(-g))
    size = np.concatenate([np.abs(one * host(da) * u) * terms, np.abs(eh[:, F:])], 1)
    assert dh.dtype == da.dtype and act.dtype == da.dtype
    close(dh, eh, dt, size)
    close(act, ea, dt)
    if weighted:
        total = np.abs(host(da) * X.swiglu(h)).sum(1)
        assert drow.dtype == torch.float32
        assert (np.abs(host(drow) - er) <= (REL + F * 2.0**-24) * total + 2.0**-110).all()
    else:
        assert drow is None
    only, none, _ = bsmm.bsmm_swiglu_backward(da, q, s, row_scale=dev(r) if weighted else None,
                                              act=False)
    assert none is None and torch.equal(only, dh)


def test_gate_gradient_against_differences():
    """The gradient of the values a checkpoint stands for, by central
    differences of the oracle's gate."""
    rng = np.random.default_rng(3)
    q, s = bsmm.bsmm_quant_int8_mx(dev(rng.standard_normal((4, 128)) * 3, torch.float32))
    h = X.restore(host(q), host(s))
    da = rng.standard_normal((4, 64)).astype(np.float32)
    dh = host(bsmm.bsmm_swiglu_backward(dev(da), q, s)[0])
    # a central difference of step d errs by d^2/6 of the third derivative (of
    # silu below 0.4) and 2^-52 |f| / d
    step = 1e-5
    for half in (0, 64):
        d = np.zeros_like(h)
        d[:, half:half + 64] = step
        slope = (X.swiglu(h + d) - X.swiglu(h - d)) / (2 * step) * da
        room = np.abs(da) * (step**2 * np.abs(h).max() + 2.0**-50 * np.abs(h).max()**2 / step)
        g = np.abs(h[:, :64]) + 1
        size = np.abs(da) * g * (np.abs(h[:, 64:]) if half == 0 else 1.0)
        assert (np.abs(dh[:, half:half + 64] - slope) <= room + 12 * 2.0**-23 * size).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gate_special_values(dt):
    h = torch.ones(3, 128, device=DEV, dtype=TDT[dt])
    h[0, 3], h[1, 70] = float("nan"), float("inf")
    a, q, s = bsmm.bsmm_swiglu(h, checkpoint=True)
    bad = np.zeros((3, 64), bool)
    bad[0, 3] = bad[1, 6] = True
    assert not np.isfinite(host(a)[bad]).any() and np.isfinite(host(a)[~bad]).all()
    da = torch.ones(3, 64, device=DEV, dtype=TDT[dt])
    r = torch.ones(3, device=DEV)
    dh, act, drow = (host(t) for t in bsmm.bsmm_swiglu_backward(da, q, s, row_scale=r))
    assert np.isnan(drow[:2]).all() and np.isfinite(drow[2])
    # row 0: gates 0..31 are NaN; row 1: ups 0..31 are, which the ups' own gradient does not use
    for row in (0, 1):
        assert np.isnan(act[row, :32]).all() and np.isfinite(act[row, 32:]).all()
        assert np.isnan(dh[row, :32]).all() and np.isfinite(dh[row, 32:64]).all()
    assert np.isnan(dh[0, 64:96]).all() and np.isfinite(dh[0, 96:]).all()
    assert np.isfinite(dh[1, 64:]).all() and np.isfinite(dh[2]).all()


def test_empty_sizes():
    z = torch.zeros
    q, s = bsmm.bsmm_quant_int8_mx(z(0, 64, device=DEV))
    assert q.shape == (0, 64) and s.shape == (0, 2)
    a, q, s = bsmm.bsmm_swiglu(z(0, 64, device=DEV), checkpoint=True)
    assert a.shape == (0, 32)
    dh, act, drow = bsmm.bsmm_swiglu_backward(a, q, s, row_scale=z(0, device=DEV))
    assert dh.shape == (0, 64) and act.shape == (0, 32) and drow.shape == (0,)
    e = z(3, 0, device=DEV)
    _, _, drow = bsmm.bsmm_swiglu_backward(e, e.to(torch.int8), e.to(torch.uint8),
                                           row_scale=torch.ones(3, device=DEV))
    assert not host(drow).any()


def test_other_stream_and_graph():
    h = gate_input(40, 96, "bf16", 1)
    da = dev(np.random.default_rng(2).standard_normal((40, 96)), torch.bfloat16)
    r = torch.rand(40, device=DEV)

    def all_of_it():
        a, q, s = bsmm.bsmm_swiglu(h, checkpoint=True)
        return (a, q, s, *bsmm.bsmm_swiglu_backward(da, q, s, row_scale=r),
                *bsmm.bsmm_quant_int8_mx(h, values=True))

    want = [host(t) for t in all_of_it()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = all_of_it()
    s.synchronize()
    assert all(np.array_equal(host(a), b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        static = all_of_it()
    for i in range(3):
        h.copy_(gate_input(40, 96, "bf16", 2 + i))
        graph.replay()
        torch.cuda.synchronize()
        got = [host(t) for t in static]
        assert all(np.array_equal(a, host(b)) for a, b in zip(got, all_of_it())), i
