"""The training example: that it runs, and its gradients.

In fp32, against 64-bit autograd of the same layer whose backward pass starts
from the values that the 8-bit checkpoints stand for: each of the at most four
products on a path sums at most 256 terms in fp32 and is off by at most 256 *
2^-23 of the sum of their magnitudes, which for terms of random sign is about
sqrt(256) times the result's size: 4 * 256 * 2^-23 * 16 = 2e-3 of the result in
the Frobenius norm at most (and 256 times less where the errors are independent).
"""

import importlib.util
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsmm
from oracle import expert as X

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PATH = os.path.join(ROOT, "examples", "moe_training.py")
LIMIT = 2e-3


@pytest.fixture(autouse=True)
def _lib(gpu_lib):
    yield


def example():
    spec = importlib.util.spec_from_file_location("moe_training", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_runs():
    r = subprocess.run([sys.executable, PATH], capture_output=True, text=True, timeout=110)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.count("step") == 3


def near(got, want, what):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    err = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert err <= LIMIT, (what, err)


@pytest.mark.parametrize("T,D,F,E,k", [(40, 96, 64, 6, 2), (1, 64, 32, 4, 3), (200, 256, 128, 8, 2)])
def test_gradients_fp32(T, D, F, E, k):
    m = example()
    layer = m.MoeLayer(D, F, E, k, alpha=0.05, dtype=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, D, device="cuda", generator=g)
    dout = torch.randn(T, D, device="cuda", generator=g)
    mask = torch.rand(T, device="cuda", generator=g) < 0.9
    mask[0] = True
    out, loss, saved = layer.forward(x, mask=mask)
    dx, d_router, d_in, d_out = layer.backward(saved, dout)
    torch.cuda.synchronize()

    logits, r, _, x8, x_scale, h8, h_scale = saved
    host = [t.double().cpu().numpy() for t in (x, layer.w_in, layer.w_out, layer.router, dout)]
    xh, w_in, w_out, router, dh_out = host
    order, offsets = r.order.cpu().numpy(), r.offsets.cpu().numpy()
    weight = r.weight.double().cpu().numpy().reshape(-1)

    # forward, in 64 bits
    h = X.expert_mm(xh, w_in, order, offsets, k)
    y = X.expert_mm(X.swiglu(h), w_out, order, offsets, 1, weight)
    near(out, y.reshape(T, k, D).sum(1), "out")
    assert not out[~mask].any()

    # backward, from what the checkpoints stand for
    hv = X.restore(h8.cpu().numpy(), h_scale.cpu().numpy())
    xv = X.restore(x8.cpu().numpy(), x_scale.cpu().numpy())
    da = X.expert_mm(dh_out, w_out.transpose(0, 2, 1), order, offsets, k)
    dh, act, dweight = X.swiglu_backward(da, hv, weight)
    near(d_out, X.expert_wgrad(dh_out, act, order, offsets, k, 1), "w_out")
    near(d_in, X.expert_wgrad(dh, xv, order, offsets, 1, k), "w_in")
    # the router: softmax over the live tokens, weights that sum to one
    lt = torch.tensor(xh @ router.T, requires_grad=True)
    index = r.index.cpu().long()
    live = mask.cpu()
    p = torch.softmax(lt[live], 1)
    picked = p.gather(1, index[live])
    wt = picked / picked.sum(1, keepdim=True)
    counts = torch.tensor(r.counts.cpu().numpy(), dtype=torch.float64)
    L = int(live.sum())
    balance = 0.05 * E / (k * L * L) * (counts * p.sum(0)).sum()
    total = (wt * torch.tensor(dweight.reshape(T, k))[live]).sum() + balance
    total.backward()
    dl = lt.grad.numpy()
    assert abs(loss.item() - balance.item()) <= 1e-5 * balance.item()
    near(d_router, dl.T @ xv, "router")
    dxs = X.expert_mm(dh, w_in.transpose(0, 2, 1), order, offsets).reshape(T, k, D).sum(1)
    near(dx, dxs + dl @ router, "x")


def test_gradient_against_differences():
    """The task's loss as a function of one expert's weights, by central
    differences in 64 bits: the gradient is that of the stored values, so it
    is compared where the checkpoint is exact (h and x of few bits)."""
    m = example()
    T, D, F, E, k = 24, 32, 32, 3, 1
    layer = m.MoeLayer(D, F, E, k, alpha=0.0, dtype=torch.float32)
    rng = np.random.default_rng(5)
    x = rng.integers(-2, 3, (T, D)).astype(np.float32)
    # one entry a row, a power of two: every h is one element of x times it
    w_in = np.zeros((E, 2 * F, D), np.float32)
    for e in range(E):
        w_in[e, np.arange(2 * F), rng.integers(0, D, 2 * F)] = 0.5
    layer.w_in.copy_(torch.from_numpy(w_in))
    dout = rng.standard_normal((T, D)).astype(np.float32)
    out, _, saved = layer.forward(torch.from_numpy(x).cuda())
    _, _, d_in, d_out = layer.backward(saved, torch.from_numpy(dout).cuda())
    r = saved[1]
    order, offsets = r.order.cpu().numpy(), r.offsets.cpu().numpy()
    weight = r.weight.double().cpu().numpy().reshape(-1)
    w_out = layer.w_out.double().cpu().numpy()

    def loss(wi, wo):
        a = X.swiglu(X.expert_mm(x, wi, order, offsets))
        return (X.expert_mm(a, wo, order, offsets, 1, weight) * dout).sum()

    step = 1e-4
    for which, grad in ((0, d_in), (1, d_out)):
        w = [w_in.astype(np.float64), w_out]
        g = grad.double().cpu().numpy()
        for _ in range(12):
            at = tuple(int(rng.integers(0, n)) for n in g.shape)
            d = np.zeros_like(w[which])
            d[at] = step
            up, dn = ([a + s * d if i == which else a for i, a in enumerate(w)] for s in (1, -1))
            slope = (loss(*up) - loss(*dn)) / (2 * step)
            # the difference: step^2 / 6 of a third derivative of a sum of T terms of size
            # 10 at most, and 2^-52 of the loss over the step; the gradient: fp32 sums
            size = np.abs(g).max()
            assert abs(slope - g[at]) <= 10 * T * step**2 + 1e-9 / step + LIMIT * size, (which, at)


def test_bfloat16_runs_and_is_near():
    """bf16: every stored activation and gradient is rounded to 2^-8 of itself
    or better, and at most 6 of them are on a path: 6 * 2^-8 = 2.3 % of the
    fp32 layer's gradients in the Frobenius norm, the checkpoints' steps of
    2^-6 of a block's maximum (an error of 2^-7, 1.5 % of a block's elements
    of a third of it) as much again in either."""
    m = example()
    T, D, F, E, k = 300, 128, 64, 4, 2
    one, two = (m.MoeLayer(D, F, E, k, dtype=dt) for dt in (torch.float32, torch.bfloat16))
    one.w_in.copy_(two.w_in)
    one.w_out.copy_(two.w_out)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(T, D, device="cuda", generator=g).to(torch.bfloat16)
    dout = torch.randn(T, D, device="cuda", generator=g).to(torch.bfloat16)
    a, _, sa = one.forward(x.float())
    b, _, sb = two.forward(x)
    assert torch.equal(sa[1].index, sb[1].index)
    for p, q in zip((a, *one.backward(sa, dout.float())), (b, *two.backward(sb, dout))):
        assert ((p - q).norm() / p.norm()).item() <= 6 * 2.0**-8 + 2 * 0.023


def test_captured_step():
    """Forward and backward in one graph, replayed on changed inputs between
    eager steps of another size."""
    m = example()
    T, D, F, E, k = 150, 128, 96, 5, 2
    layer = m.MoeLayer(D, F, E, k)
    x = torch.randn(T, D, device="cuda").to(torch.bfloat16)
    dout = torch.randn(T, D, device="cuda").to(torch.bfloat16)

    def step():
        out, loss, saved = layer.forward(x)
        return (out, loss, *layer.backward(saved, dout))

    step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        static = step()
    big = torch.randn(900, D, device="cuda").to(torch.bfloat16)
    for _ in range(3):
        x.copy_(torch.randn(T, D, device="cuda"))
        dout.copy_(torch.randn(T, D, device="cuda"))
        graph.replay()
        out, _, saved = layer.forward(big)
        layer.backward(saved, big)
        torch.cuda.synchronize()
        for a, b in zip(static, step()):
            assert torch.equal(a, b)
