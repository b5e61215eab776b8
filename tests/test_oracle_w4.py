"""The 4-bit oracle pinned on hand-worked groups, and against plain loops."""

import numpy as np
import pytest

from oracle import w4


def test_symmetric_group_by_hand():
    w = np.zeros((1, 32), np.float32)
    w[0, :6] = [7.0, -7.0, 2.5, -2.5, 3.5, 0.49]
    code, s, z, v = w4.quantise(w, 32)
    assert s[0, 0] == 1.0 and z[0, 0] == 8
    # halves go to the even integer
    assert code[0, :7].tolist() == [15, 1, 10, 6, 12, 8, 8]
    assert v[0, :7].tolist() == [7, -7, 2, -2, 4, 0, 0]


def test_zero_point_group_by_hand():
    w = np.zeros((1, 32), np.float32)
    w[0, :4] = [10.0, -5.0, 1.0, 9.5]
    code, s, z, v = w4.quantise(w, 32, symmetric=False)
    assert s[0, 0] == 1.0 and z[0, 0] == 5
    assert code[0, :5].tolist() == [15, 0, 6, 15, 5]        # 9.5 -> 10 (even)
    assert v[0, :5].tolist() == [10, -5, 1, 10, 0]
    # one-sided groups keep 0 in range
    code, s, z, v = w4.quantise(np.full((1, 32), 3.0, np.float32), 32, symmetric=False)
    assert z[0, 0] == 0 and (code == 15).all() and abs(v[0, 0] - 3.0) < 1e-6


@pytest.mark.parametrize("sym", [True, False])
def test_empty_group(sym):
    for tiny in (0.0, 1e-45):
        code, s, z, v = w4.quantise(np.full((2, 64), tiny, np.float32), 64, sym)
        assert (s == 1.0).all() and (v == 0.0).all() and (code == (8 if sym else 0)).all()
        assert (z == (8 if sym else 0)).all()


def test_bf16_rounding():
    import torch
    rng = np.random.default_rng(3)
    bits = rng.integers(0, 0x7F000000, 20000, dtype=np.uint32)
    bits[:3] = [1, 0x00008000, 0x00018000]                  # subnormals, a tie each way
    a = bits.view(np.float32)
    want = torch.from_numpy(a).to(torch.bfloat16).double().numpy()
    assert np.array_equal(w4.bf16(a.astype(np.float64)), want)


def test_pack_round_trip():
    code = np.random.default_rng(1).integers(0, 16, (5, 64))
    q = w4.pack(code)
    assert q.shape == (5, 32) and q[0, 0] == code[0, 0] + 16 * code[0, 1]
    assert np.array_equal(w4.unpack(q), code)


def test_products_against_loops():
    rng = np.random.default_rng(2)
    code = rng.integers(0, 16, (2, 3, 64))
    q = np.stack([w4.pack(c) for c in code])
    s, z = rng.random((2, 3, 2)), rng.integers(0, 16, (2, 3, 2))
    x = rng.standard_normal((4, 64))
    order, offsets = np.array([5, 0, 3, 1, 7, 2, 4, 6]), [0, 3, 6]
    rs = rng.random(8)
    y = w4.w4_expert_mm(x, q, s, z, order, offsets, slots_per_row=2, row_scale=rs)
    for i, slot in enumerate(order):
        for n in range(3):
            e = 0 if i < 3 else 1
            t = sum((code[e, n, k] - z[e, n, k // 32]) * s[e, n, k // 32] * x[slot // 2, k]
                    for k in range(64)) * rs[slot] if i < 6 else 0.0
            assert abs(y[slot, n] - t) < 1e-12
    assert np.allclose(w4.w4_mm(x, q[0], s[0], z[0]),
                       w4.w4_expert_mm(x, q[:1], s[:1], z[:1], np.arange(4), [0, 4]))
