"""Products of routed rows with their experts' weights, 8-bit checkpoints and
the gate, written from their definitions in 64 bits (oracle; test
infrastructure: the library shares no code with it).

A slot is one (token, choice) pair; ``order`` lists the slots by expert and
``offsets`` says where each expert's run begins and ends.
"""

from __future__ import annotations

import numpy as np


def slots_of(order, offsets, e, S):
    """The slots of expert e (order None: slot i at position i)."""
    run = np.arange(offsets[e], offsets[e + 1])
    return run if order is None else np.asarray(order)[run]


def expert_mm(x, w, order, offsets, slots_per_row=1, row_scale=None):
    """out[s] = row_scale[s] * w[e] x[s // slots_per_row]; 0 without an expert."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    S = x.shape[0] * slots_per_row if order is None else len(order)
    out = np.zeros((S, w.shape[1]))
    for e in range(w.shape[0]):
        for s in slots_of(order, offsets, e, S):
            out[s] = w[e] @ x[s // slots_per_row]
            if row_scale is not None:
                out[s] *= row_scale[s]
    return out


def expert_wgrad(dy, x, order, offsets, dy_slots_per_row=1, x_slots_per_row=1):
    """dw[e] = sum over e's slots of the outer product of dy's and x's row."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    E = len(offsets) - 1
    S = dy.shape[0] * dy_slots_per_row if order is None else len(order)
    dw = np.zeros((E, dy.shape[1], x.shape[1]))
    for e in range(E):
        s = slots_of(order, offsets, e, S).astype(np.int64)
        dw[e] = dy[s // dy_slots_per_row].T @ x[s // x_slots_per_row]
    return dw


def quantise(x):
    """An 8-bit checkpoint of x [R, K]: int8 codes, a byte per 32 elements,
    the values (NaN in a block that holds a NaN or an infinity)."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[0], -1, 32)
    bad = ~np.isfinite(b).all(2)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(2) if b.size else np.zeros(b.shape[:2])
    p = np.frexp(top)[1] - 1                      # top = m 2^p, m in [1, 2)
    byte = np.where(top == 0.0, 127, np.maximum(p + 127, 0))
    q = np.rint(np.ldexp(b, (133 - byte)[..., None]))
    q = np.clip(q, -127, 127)
    byte = np.where(bad, 255, byte)
    q = q.reshape(x.shape).astype(np.int8)
    return q, byte.astype(np.uint8), restore(q, byte)


def restore(q, byte):
    """What a checkpoint stands for."""
    byte = np.asarray(byte, np.int64)
    step = np.where(byte == 255, np.nan, np.ldexp(1.0, np.minimum(byte, 254) - 133))
    return np.asarray(q, np.float64) * np.repeat(step, 32, axis=-1)


def sigmoid(g):
    with np.errstate(over="ignore"):
        return np.where(g >= 0, 1 / (1 + np.exp(-np.abs(g))),
                        np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))


def swiglu(h):
    """silu(first half) * second half."""
    h = np.asarray(h, np.float64)
    F = h.shape[1] // 2
    g, u = h[:, :F], h[:, F:]
    return g * sigmoid(g) * u


def swiglu_backward(da, h, row_scale=None):
    """(dh, row_scale * swiglu(h), row_scale's gradient) for da, the gradient
    of row_scale * swiglu(h)."""
    da, h = np.asarray(da, np.float64), np.asarray(h, np.float64)
    F = h.shape[1] // 2
    g, u = h[:, :F], h[:, F:]
    r = np.ones((len(da), 1)) if row_scale is None else np.asarray(row_scale, np.float64)[:, None]
    s = sigmoid(g)
    dg = r * da * u * s * (1 + g * sigmoid(-g))
    return (np.concatenate([dg, r * da * g * s], 1), r * g * s * u, (da * g * s * u).sum(1))
