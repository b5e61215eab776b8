"""Pins of the oracle of the experts' products, checkpoints and gate (CPU)."""

from fractions import Fraction

import numpy as np
import torch

from exact import floor_log2, rne
from oracle import expert as X


def test_products_by_hand():
    x = np.array([[1.0, 2.0], [3.0, 5.0]])
    w = np.arange(12.0).reshape(2, 3, 2)
    # tokens x 2 choices: slots 0..3; expert 0 has slots 3 and 0, expert 1 slot 1, slot 2 none
    order, offsets = np.array([0, 3, 1, 2]), np.array([0, 2, 3])
    out = X.expert_mm(x, w, order, offsets, 2, np.array([1.0, 2.0, 7.0, 0.5]))
    assert out[0].tolist() == [2.0, 8.0, 14.0]          # w[0] x[0]
    assert out[1].tolist() == [40.0, 52.0, 64.0]        # 2 w[1] x[0]
    assert out[2].tolist() == [0.0, 0.0, 0.0]
    assert out[3].tolist() == [2.5, 10.5, 18.5]         # w[0] x[1] / 2
    dw = X.expert_wgrad(np.arange(12.0).reshape(4, 3), x, order, offsets, 1, 2)
    # slot 0: dy (0, 1, 2), token 0; slot 3: dy (9, 10, 11), token 1
    assert dw[0].tolist() == [[27.0, 45.0], [31.0, 52.0], [35.0, 59.0]]
    assert dw[1].tolist() == [[3.0, 6.0], [4.0, 8.0], [5.0, 10.0]]


def test_wgrad_is_the_products_gradient():
    rng = np.random.default_rng(3)
    x = torch.tensor(rng.standard_normal((5, 7)), requires_grad=True)
    w = torch.tensor(rng.standard_normal((3, 4, 7)), requires_grad=True)
    order, offsets = rng.permutation(10), np.array([0, 4, 4, 9])
    dy = rng.standard_normal((10, 4))
    total = 0.0
    for e in range(3):
        for s in order[offsets[e]:offsets[e + 1]]:
            total = total + (torch.tensor(dy[s]) * (w[e] @ x[s // 2])).sum()
    total.backward()
    got = X.expert_wgrad(dy, x.detach().numpy(), order, offsets, 1, 2)
    assert np.allclose(got, w.grad.numpy(), rtol=1e-13, atol=1e-13)
    dx = X.expert_mm(dy, w.detach().numpy().transpose(0, 2, 1), order, offsets)
    assert np.allclose(dx.reshape(5, 2, 7).sum(1), x.grad.numpy(), rtol=1e-13, atol=1e-13)


def test_checkpoint_against_fractions():
    rng = np.random.default_rng(4)
    x = (rng.standard_normal((6, 64)) * np.exp2(rng.integers(-140, 120, (6, 1)))).astype(np.float32)
    x[0, :32] = 0.0
    x[1, 3] = 0.0
    x[2, :32] = np.arange(32) + 0.5                     # ties; 31.5 in steps of 1/4
    x[3, :32] = 1.999                                   # beyond the largest code
    q, byte, values = X.quantise(x)
    for r in range(6):
        for b in range(2):
            v = [Fraction(float(t)) for t in x[r, 32 * b:32 * b + 32]]
            top = max(abs(t) for t in v)
            want = 127 if top == 0 else max(floor_log2(top) + 127, 0)
            assert byte[r, b] == want
            for i, t in enumerate(v):
                n = rne(t / Fraction(2) ** (want - 133), 60, 0) if t else Fraction(0)
                # quantum 2^-59 at exponent 0 is no rounding: to integers by hand
                n = Fraction(round(n))
                n = max(min(n, 127), -127)
                k = 32 * b + i
                assert q[r, k] == n
                assert Fraction(float(values[r, k])) == n * Fraction(2) ** (want - 133)
                assert abs(Fraction(float(values[r, k])) - t) <= Fraction(2) ** (want - 133)


def test_checkpoint_special_blocks():
    x = np.ones((1, 96))
    x[0, 5], x[0, 40] = np.inf, np.nan
    q, byte, values = X.quantise(x)
    assert byte.tolist() == [[255, 255, 127]]
    assert not q[0, :64].any() and (q[0, 64:] == 64).all()
    assert np.isnan(values[0, :64]).all() and (values[0, 64:] == 1.0).all()


def test_gate_gradient():
    rng = np.random.default_rng(5)
    h = torch.tensor(rng.standard_normal((3, 12)) * 4, requires_grad=True)
    r = torch.tensor(rng.random(3), requires_grad=True)
    da = torch.tensor(rng.standard_normal((3, 6)))
    a = torch.nn.functional.silu(h[:, :6]) * h[:, 6:]
    (da * r[:, None] * a).sum().backward()
    dh, act, drow = X.swiglu_backward(da.numpy(), h.detach().numpy(), r.detach().numpy())
    assert np.allclose(dh, h.grad.numpy(), rtol=1e-13, atol=1e-15)
    assert np.allclose(drow, r.grad.numpy(), rtol=1e-13)
    assert np.allclose(act, (r[:, None] * a).detach().numpy(), rtol=1e-14)
    assert np.allclose(X.swiglu(h.detach().numpy()), a.detach().numpy(), rtol=1e-14)
    # against differences
    step = 1e-6
    for k in range(12):
        d = np.zeros((3, 12))
        d[:, k] = step
        up, dn = (X.swiglu(h.detach().numpy() + s * d) for s in (1, -1))
        slope = (r.detach().numpy()[:, None] * da.numpy() * (up - dn)).sum(1) / (2 * step)
        assert np.allclose(slope, dh[:, k], rtol=1e-7, atol=1e-8)
