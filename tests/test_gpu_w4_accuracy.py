"""The 4-bit products on activations whose sum is far larger than their
product with the weight: of one sign, with a mean, with one large channel
that meets only weights of 0.  Both kernels, one limit.

Every product (code - zero) x is exact, so the error is that of the fp32
additions: over a group of G elements at most P G of them (P: 3 parts of fp32
activations, else 1), each off by at most 2**-23 of the partial sum and
towards 0, 2**-24 on average.  Weights of mean 0 give the terms random signs,
so the partial sum of g terms is sqrt(g / G) of the group's, and the additions
of a group lose 2/3 P G 2**-24 of it.  Adding K / G groups errs by 2**-24 of
the sum each, independently.  Together (2/3 P G + sqrt(K / G)) 2**-24 in the
Frobenius norm, and an element 10 times that of the result's rms.
"""

import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsmm
from oracle import w4

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TDT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _lib(gpu_lib):
    yield


def activations(kind, M, K, rng):
    x = rng.standard_normal((M, K))
    if kind == "one sign":
        x = np.abs(x)
    elif kind == "mean":
        x += 5.0
    else:
        x[:, 7] = 3000.0 * (1.0 + rng.random(M))
    return x.astype(np.float32)


def operands(kind, lead, K, group, sym, seed):
    w = np.random.default_rng(seed).standard_normal((*lead, K)).astype(np.float32) * 0.02
    if kind == "channel":
        w[..., 7] = 0.0
    return bsmm.bsmm_quant_w4(torch.from_numpy(w).to(DEV), group=group, symmetric=sym)


def host(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def check(got, want, K, group, dt):
    tol = (2 / 3 * (3 if dt == "f32" else 1) * group + (K / group) ** 0.5) * 2.0**-24
    err = np.abs(host(got) - want)
    off = np.linalg.norm(err) / np.linalg.norm(want)
    assert off <= tol, f"{off:.1e} of {tol:.1e}"
    assert err.max() <= 10 * tol * np.sqrt((want ** 2).mean())


@pytest.mark.parametrize("kind", ["one sign", "mean", "channel"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("group,sym", [(128, True), (128, False), (32, True), (64, False)])
def test_products(kind, dt, group, sym):
    N, K = 2100, 1024
    q, s, z = operands(kind, (N,), K, group, sym, group)
    x = torch.from_numpy(activations(kind, 2048, K, np.random.default_rng(1))).to(DEV, TDT[dt])
    want = w4.w4_mm(host(x), host(q), host(s), None if sym else host(z))
    # 1 to 40 rows on the kernel of few rows, 2048 on tiles
    assert bsmm.bsmm_w4_workspace_bytes("f32", 1, 40, 40, N, K, group) == 0
    assert bsmm.bsmm_w4_workspace_bytes("f32", 1, 2048, 2048, N, K, group) > 0
    for M in (1, 13, 40, 2048):
        check(bsmm.bsmm_w4_mm(x[:M], q, s, z, out_dtype="f32"), want[:M], K, group, dt)


@pytest.mark.parametrize("kind", ["one sign", "mean", "channel"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 24])
def test_experts(kind, dt, T):
    E, N, K, k, group = 8, 96, 2048, 4, 128
    q, s, z = operands(kind, (E, N), K, group, False, 5)
    rng = np.random.default_rng(T)
    x = torch.from_numpy(activations(kind, T, K, rng)).to(DEV, TDT[dt])
    r = bsmm.bsmm_route_topk(torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32))
                             .to(DEV), k)
    got = bsmm.bsmm_w4_expert_mm(x, q, s, z, r.order, r.offsets, slots_per_row=k, out_dtype="f32")
    want = w4.w4_expert_mm(host(x), host(q), host(s), host(z), host(r.order), host(r.offsets), k)
    check(got, want, K, group, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_zero_points_of_a_whole_byte(dt, group):
    """Zero points are bytes: 0 to 255, integers and sums below 2**24."""
    N, K = 2100, 512
    rng = np.random.default_rng(group)
    q = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    z = rng.integers(0, 256, (N, K // group)).astype(np.uint8)
    s = np.ones((N, K // group), np.float32)
    x = rng.integers(-3, 4, (2048, K)).astype(np.float32)
    want = w4.w4_mm(x, q, s, z)
    dx = torch.from_numpy(x).to(DEV, TDT[dt])
    ops = [torch.from_numpy(t).to(DEV) for t in (q, s, z)]
    for M in (1, 13, 40, 2048):
        got = bsmm.bsmm_w4_mm(dx[:M], *ops, out_dtype="f32")
        assert np.array_equal(host(got), want[:M])
