"""4-bit weights, written from their definition in 64 bits (oracle; test
infrastructure: the library shares no code with it).

A weight [R, K] is kept as codes 0..15 with one scale, and optionally one
zero point, per group of consecutive elements of a row:
``value = (code - zero) * scale``.  Two codes share a byte along K, the low
nibble holding the even element.

Readings: every quotient (``amax / 7``, ``(hi - lo) / 15``, ``w / scale``,
``-lo / scale``) and ``hi - lo`` is one correctly rounded binary32 operation;
a bf16 scale is rounded to nearest even before it divides.  The binary32
quotient of two binary32 numbers is their binary64 quotient rounded to
binary32 (53 >= 2 * 24 + 2 bits make the second rounding innocuous).  A group
whose scale is 0 gets scale 1, zero point 0 (8 where none are kept) and codes
equal to it.
"""

from __future__ import annotations

import numpy as np


def f32(a):
    """Nearest binary32, as binary64 values."""
    return np.asarray(a, np.float64).astype(np.float32).astype(np.float64)


def bf16(a):
    """Nearest bfloat16 (ties to even) of binary32 values, as binary64."""
    a = np.asarray(a, np.float64)
    m, e = np.frexp(a)
    step = np.ldexp(1.0, np.maximum(e - 8, -133))
    return np.where(a == 0.0, a, np.rint(a / step) * step)


def pack(code):
    """Codes [R, K] -> bytes [R, K/2]."""
    code = np.asarray(code, np.uint8)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)


def unpack(q):
    q = np.asarray(q, np.uint8)
    out = np.empty(q.shape[:-1] + (2 * q.shape[-1],), np.int64)
    out[..., 0::2] = q % 16
    out[..., 1::2] = q // 16
    return out


def quantise(w, group, symmetric=True, scale_type="f32"):
    """(codes [R, K], scale [R, K/group], zero [R, K/group], values [R, K])
    of binary32 values w; zero is 8 everywhere for the symmetric form."""
    w = np.asarray(w, np.float64)
    R, K = w.shape
    f = w.reshape(R, K // group, group)
    if symmetric:
        s = f32(np.abs(f).max(2) / 7.0)
    else:
        lo, hi = np.minimum(f.min(2), 0.0), np.maximum(f.max(2), 0.0)
        s = f32(f32(hi - lo) / 15.0)
    if scale_type == "bf16":
        s = bf16(s)
    none = s == 0.0
    s = np.where(none, 1.0, s)
    n = np.rint(f32(f / s[..., None]))
    if symmetric:
        z = np.full(s.shape, 8.0)
        code = np.clip(n, -8, 7) + 8
    else:
        z = np.where(none, 0.0, np.clip(np.rint(f32(-lo / s)), 0, 15))
        code = np.clip(n + z[..., None], 0, 15)
    code = np.where(none[..., None], z[..., None], code)
    values = f32((code - z[..., None]) * s[..., None]).reshape(R, K)
    return code.reshape(R, K).astype(np.uint8), s, z.astype(np.uint8), values


def dequantise(q, scale, zero=None):
    """Bytes [N, K/2] with scale / zero [N, KG] -> values [N, K], 64 bits."""
    code = unpack(q)
    N, K = code.shape
    KG = scale.shape[1]
    z = np.full((N, KG), 8, np.int64) if zero is None else np.asarray(zero, np.int64)
    v = (code.reshape(N, KG, K // KG) - z[..., None]) * np.asarray(scale, np.float64)[..., None]
    return v.reshape(N, K)


def w4_mm(x, q, scale, zero=None):
    return np.asarray(x, np.float64) @ dequantise(q, scale, zero).T


def w4_expert_mm(x, q, scale, zero, order, offsets, slots_per_row=1, row_scale=None):
    """x [R, K], q [E, N, K/2], order [S], offsets [E + 1] -> [S, N]."""
    order = np.asarray(order)
    y = np.zeros((order.size, q.shape[1]))
    for e in range(q.shape[0]):
        slots = order[offsets[e]:offsets[e + 1]]
        if slots.size:
            y[slots] = w4_mm(np.asarray(x, np.float64)[slots // slots_per_row], q[e], scale[e],
                             None if zero is None else zero[e])
    return y if row_scale is None else y * np.asarray(row_scale, np.float64)[:, None]
