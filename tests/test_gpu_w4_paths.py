"""The 4-bit products on every kernel and address path, each named and
checked to be the one that the sizes take: integers with power-of-two scales,
whose sums are exact in any order, and normal data within the products' limit.
"""

import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsmm
from oracle import w4
from test_gpu_w4 import DEV, TDT, close, dev, host, integer_case, routing, same

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(gpu_lib):
    yield


def long_row(group):
    """An odd number of groups, and for groups of 32 a last chunk of one."""
    return {32: 672, 64: 704, 128: 640}[group]


# scale type, zero points, output type
KINDS = [("f32", True, "f32"), ("bf16", False, "bf16"), ("bf16", True, "f32"),
         ("f32", False, "f32")]


@pytest.mark.parametrize("kernel,M,N", [("rows4", 1, 257), ("rows4", 4, 33), ("rows16", 13, 257),
                                        ("rows32", 41, 257), ("tile128", 1290, 2500),
                                        ("tile256", 2047, 2100)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_dense(kernel, M, N, group, dt):
    K = long_row(group)
    if dt == "f32" and kernel == "rows32":
        kernel = "rows16"
    assert bsmm.bsmm_w4_plan_name(dt, False, 1, M, M, N, K, group) == kernel
    for i, (st, zero, out) in enumerate(KINDS):
        c = integer_case(M, N, K, group, zero, dt, i)
        y = bsmm.bsmm_w4_mm(dev(c["x"], TDT[dt]), dev(c["q"]), dev(c["s"], TDT[st]),
                            dev(c["z"]) if zero else None, out_dtype=out)
        same(y, w4.w4_mm(c["x"], c["q"], c["s"], c["z"]), out)


@pytest.mark.parametrize("kernel,T,k,E,N", [("rows4", 1, 8, 64, 40), ("rows4", 9, 2, 9, 129),
                                            ("rows16", 33, 4, 16, 40), ("rows32", 100, 4, 8, 70),
                                            ("tile128", 700, 4, 8, 1500)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_routed(kernel, T, k, E, N, group, dt):
    K = long_row(group)
    if dt == "f32" and kernel == "rows32":
        kernel = "rows16"
    for i, (st, zero, out) in enumerate(KINDS):
        second = i % 2 == 1
        R = T * k if second else T
        assert bsmm.bsmm_w4_plan_name(dt, True, E, R, T * k, N, K, group) == kernel
        order, offsets = routing(T, k, E, i, 0.3 if i == 2 else 0.0)
        c = integer_case(R, N, K, group, zero, dt, i, E)
        rs = np.exp2(np.random.default_rng(i).integers(-2, 2, T * k)).astype(np.float32)
        y = bsmm.bsmm_w4_expert_mm(
            dev(c["x"], TDT[dt]), dev(c["q"]), dev(c["s"], TDT[st]),
            dev(c["z"]) if zero else None, dev(order), dev(offsets),
            slots_per_row=1 if second else k, row_scale=dev(rs) if second else None,
            out_dtype=out)
        same(y, w4.w4_expert_mm(c["x"], c["q"], c["s"], c["z"], order, offsets,
                                1 if second else k, rs if second else None), out)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("st,group", [("bf16", 128), ("f32", 32)])
def test_routed_tiles_normal_data(dt, st, group):
    T, k, E, N, K = 700, 4, 8, 1500, 1024
    assert bsmm.bsmm_w4_plan_name(dt, True, E, T, T * k, N, K, group) == "tile128"
    rng = np.random.default_rng(group)
    order, offsets = routing(T, k, E, 3)
    w = dev((rng.standard_normal((E, N, K)) * 0.02).astype(np.float32))
    q, s, z = bsmm.bsmm_quant_w4(w, group=group, symmetric=False, scale_dtype=st)
    x = dev(rng.standard_normal((T, K)).astype(np.float32), TDT[dt])
    close(lambda out: bsmm.bsmm_w4_expert_mm(x, q, s, z, dev(order), dev(offsets),
                                             slots_per_row=k, out_dtype=out),
          w4.w4_expert_mm(host(x), host(q), host(s), host(z), order, offsets, k))


def far_rows(t, ld):
    """t with the row stride ld and, of three dimensions, its blocks in order."""
    rows = t.numel() // t.shape[-1]
    wide = torch.zeros(rows * ld, dtype=t.dtype, device=DEV).view(*t.shape[:-1], ld)
    wide[..., :t.shape[-1]] = t
    return wide[..., :t.shape[-1]]


@pytest.mark.parametrize("far", ["x", "w", "scale", "zero"])
@pytest.mark.parametrize("T,K,group", [(1, 288, 32), (3, 192, 64), (3, 256, 128)])
def test_routed_rows_far_apart(far, T, K, group):
    """Row strides whose multiples pass 31 bits."""
    E, N, k = 2, 3, 2
    order, offsets = routing(T, k, E, T)
    c = integer_case(T, N, K, group, True, "bf16", K, E)
    ops = dict(x=dev(c["x"], torch.bfloat16), w=dev(c["q"]), scale=dev(c["s"]), zero=dev(c["z"]))
    ops[far] = far_rows(ops[far], {"x": 1 << 29, "w": 1 << 27, "scale": 1 << 25,
                                   "zero": 1 << 28}[far])
    if far == "x":
        assert T == 1 or T * ops["x"].stride(0) * 2 >= 1 << 31
    y = bsmm.bsmm_w4_expert_mm(ops["x"], ops["w"], ops["scale"], ops["zero"], dev(order),
                               dev(offsets), slots_per_row=k, out_dtype="f32")
    same(y, w4.w4_expert_mm(c["x"], c["q"], c["s"], c["z"], order, offsets, k), "f32")


def test_dense_in_two_launches():
    """More than 65535 workgroups of rows."""
    M, N, K = 65536 * 16 + 5, 18, 32
    c = integer_case(M, N, K, 32, True, "f32", 8)
    out = torch.full((M + 16, N), -5.0, device=DEV)
    y = bsmm.bsmm_w4_mm(dev(c["x"]), dev(c["q"]), dev(c["s"]), dev(c["z"]), out_dtype="f32",
                        out=out[:M], workspace=False)
    same(y, w4.w4_mm(c["x"], c["q"], c["s"], c["z"]), "f32")
    assert (out[M:] == -5.0).all()
