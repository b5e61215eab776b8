"""The expert router on the GPU against the 64-bit oracle.

Integers (choice, counts, offsets, order, live) must be equal.  Tolerances:
p = 2^x (1 + 2 units) / s, with s a sum of E terms in fp32 along a lane and 6
steps across lanes (at most 16 + 6 roundings, 2**-24 each) and the
difference logit - max rounded once (2**-24 of up to 30 here, an error of
30 * 2**-24 in the exponent): weights are within 64 * 2**-24 relative.
prob_sum adds at most T / 256 / 16 + 16 + 64 + 16 terms of one sign one after
another, below 256 * 2**-24 relative here, the loss a few more: 320 * 2**-24.
A gradient is p times a difference of terms no larger than |c|max and
|dw|max: 128 * 2**-24 of p (2 |c|max + 2 |dw|max) (renormalised: w for p on
the chosen experts), and bf16 adds 2**-8 of the value.
"""

import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsmm
from oracle import route as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TDT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0**-24


@pytest.fixture(autouse=True)
def _lib(gpu_lib):
    yield


def dev(a, dt=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dt is None else t.to(dt)


def host(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def logits(T, E, dt, seed, kind="normal"):
    """Values exactly representable in dt; bf16 and "ties" have many equals."""
    rng = np.random.default_rng(seed)
    l = rng.standard_normal((T, E)) * 2 + rng.standard_normal(E)
    if kind == "ties":
        l = np.round(l)
        l[l == 0] = np.where(rng.random((l == 0).sum()) < 0.5, 0.0, -0.0)
    if kind == "masked":
        l[rng.random((T, E)) < 0.5] = -np.inf
        l[rng.random(T) < 0.2] = -np.inf
        l[rng.random(T) < 0.1, 1:] = np.finfo(np.float32).min if dt == "f32" else -3.3895e38
    return host(dev(l.astype(np.float32), TDT[dt])).astype(np.float32)


def check_forward(r, want, loss=True):
    for n in ("index", "counts", "offsets", "order"):
        g = host(getattr(r, n))
        assert g.dtype == np.int32 and np.array_equal(g, want[n]), n
    w = host(r.weight)
    assert (np.abs(w - want["weight"]) <= 64 * U * want["weight"]).all()
    if not loss:
        assert r.live is None and r.prob_sum is None and r.loss is None
        return
    assert host(r.live).tolist() == [want["live"]]
    assert (np.abs(host(r.prob_sum) - want["prob_sum"]) <= 256 * U * want["prob_sum"]).all()
    assert abs(host(r.loss)[0] - want["loss"]) <= 320 * U * want["loss"]


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (3, 4, 4), (17, 60, 6), (64, 65, 3),
                                   (65, 128, 8), (63, 129, 32), (200, 256, 8), (1000, 16, 2),
                                   (130, 257, 10), (77, 512, 6), (129, 513, 2), (70, 1000, 32),
                                   (66, 1024, 1), (4097, 24, 5)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_forward(T, E, k, dt):
    for i, kind in enumerate(("normal", "ties", "masked")):
        l = logits(T, E, dt, T + E + i, kind)
        mask = np.random.default_rng(i).random(T) < 0.8 if kind == "masked" else None
        renorm = i != 1
        r = bsmm.bsmm_route_topk(dev(l, TDT[dt]), k, mask=None if mask is None else dev(mask),
                                 renorm=renorm, alpha=0.25)
        check_forward(r, R.route(l, k, mask, renorm, 0.25))


def test_forward_large():
    """More than 64 tokens to a block, the last block short."""
    T, E, k = 256 * 64 * 2 + 37, 8, 2
    l = logits(T, E, "f32", 4, "masked")
    r = bsmm.bsmm_route_topk(dev(l), k, alpha=1.0)
    check_forward(r, R.route(l, k, alpha=1.0))


@pytest.mark.parametrize("T", [1, 40, 300])
def test_forward_serving_and_strides(T):
    """No loss; rows of a wider, unaligned matrix with poison around them."""
    for dt in ("bf16", "f32"):
        l = logits(T, 37, dt, T)
        wide = torch.full((T, 45), float("nan"), device=DEV, dtype=TDT[dt])
        wide[:, 3:40] = dev(l)
        mask = (np.arange(T) % 3 != 1).astype(np.uint8)
        r = bsmm.bsmm_route_topk(wide[:, 3:40], 5, mask=dev(mask))
        check_forward(r, R.route(l, 5, mask), loss=False)


@pytest.mark.parametrize("T", [1, 70])
def test_forward_all_masked(T):
    l = logits(T, 20, "f32", 3)
    for mask, ll in ((np.zeros(T, bool), l), (None, np.full_like(l, -np.inf))):
        r = bsmm.bsmm_route_topk(dev(ll), 4, mask=None if mask is None else dev(mask), alpha=1.0)
        check_forward(r, R.route(ll, 4, mask, alpha=1.0))
        assert host(r.loss)[0] == 0.0 and (host(r.index) == -1).all()


def test_forward_no_tokens():
    r = bsmm.bsmm_route_topk(torch.empty(0, 10, device=DEV), 2, alpha=1.0)
    assert r.index.shape == (0, 2) and r.order.numel() == 0
    assert (host(r.counts) == 0).all() and (host(r.offsets) == 0).all()
    assert host(r.loss)[0] == 0.0 and host(r.live)[0] == 0 and (host(r.prob_sum) == 0).all()


@pytest.mark.parametrize("T", [4, 100])
def test_nan_and_inf(T):
    """A NaN or +inf poisons its own row's weights and the sums, nothing
    else; in a masked token it does nothing."""
    l = logits(T, 12, "f32", 9)
    l[1, 3] = np.nan
    l[2, 5] = np.inf
    mask = np.ones(T, bool)
    for renorm in (True, False):
        r = bsmm.bsmm_route_topk(dev(l), 3, mask=dev(mask), renorm=renorm, alpha=1.0)
        want = R.route(l, 3, mask, renorm, 1.0)
        for n in ("index", "counts", "offsets", "order"):
            assert np.array_equal(host(getattr(r, n)), want[n]), n
        w = host(r.weight)
        assert np.isnan(w[1:3]).all() and np.isnan(host(r.loss)[0])
        keep = [t for t in range(T) if t not in (1, 2)]
        assert (np.abs(w[keep] - want["weight"][keep]) <= 64 * U * want["weight"][keep]).all()
    mask[1:3] = False
    r = bsmm.bsmm_route_topk(dev(l), 3, mask=dev(mask), alpha=1.0)
    check_forward(r, R.route(l, 3, mask, alpha=1.0))
    d = bsmm.bsmm_route_topk_backward(dev(l), r.index, r.weight, r.counts, r.live,
                                      dweight=torch.ones_like(r.weight),
                                      dloss=torch.ones(1, device=DEV), alpha=1.0, mask=dev(mask))
    assert np.isfinite(host(d)).all() and (host(d)[1:3] == 0).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (17, 60, 6), (65, 128, 8), (33, 129, 32),
                                   (200, 256, 8), (40, 512, 6), (9, 1024, 32)])
def test_backward(T, E, k, renorm, dt):
    rng = np.random.default_rng(T + E)
    for kind in ("normal", "masked"):
        l = logits(T, E, dt, T + k, kind)
        mask = rng.random(T) < 0.8 if kind == "masked" else None
        f = R.route(l, k, mask, renorm, 0.5)
        dw, dl = rng.standard_normal((T, k)).astype(np.float32), np.float32(1.7)
        r = bsmm.bsmm_route_topk(dev(l, TDT[dt]), k, mask=None if mask is None else dev(mask),
                                 renorm=renorm, alpha=0.5)
        for use_w, use_l in ((True, True), (True, False), (False, True), (False, False)):
            out = torch.full((T, E), 5.0, device=DEV, dtype=TDT[dt])
            d = bsmm.bsmm_route_topk_backward(
                dev(l, TDT[dt]), r.index, r.weight, r.counts, r.live,
                dweight=dev(dw) if use_w else None,
                dloss=torch.tensor([dl], device=DEV) if use_l else None, alpha=0.5,
                mask=None if mask is None else dev(mask), renorm=renorm, out=out)
            want = R.gradient(l, f["index"], f["counts"], f["live"], dw * use_w, dl * use_l, 0.5,
                              mask, renorm)
            c = 1.7 * 0.5 * E / (k * max(f["live"], 1) ** 2) * f["counts"].max() * use_l
            size = 2 * c + 2 * np.abs(dw).max() * use_w
            big = np.zeros((T, E))
            for t in range(T):
                if f["index"][t, 0] >= 0 and (mask is None or mask[t]):
                    big[t] = R._softmax(l[t].astype(np.float64))
                    for j, e in enumerate(f["index"][t]):
                        if e >= 0:
                            big[t, e] = max(big[t, e], f["weight"][t, j])
            tol = 128 * U * big * size + (2.0**-8 * np.abs(want) if dt == "bf16" else 0)
            assert (np.abs(host(d) - want) <= tol).all()


def test_backward_against_differences():
    """The gradient against differences of the GPU forward pass (fp32: a
    step of 2**-6 leaves a truncation error of its square over 6 and a
    rounding error of 2**-17 of the sum)."""
    T, E, k = 6, 20, 4
    rng = np.random.default_rng(0)
    l = logits(T, E, "f32", 11)
    l += np.arange(E, dtype=np.float32)[::-1] * 0.5         # no change of choice within a step
    dw = rng.standard_normal((T, k)).astype(np.float32)
    for renorm in (True, False):
        r = bsmm.bsmm_route_topk(dev(l), k, renorm=renorm, alpha=0.5)
        d = host(bsmm.bsmm_route_topk_backward(
            dev(l), r.index, r.weight, r.counts, r.live, dweight=dev(dw),
            dloss=torch.ones(1, device=DEV), alpha=0.5, renorm=renorm))

        def f(x):
            s = bsmm.bsmm_route_topk(dev(x), k, renorm=renorm, alpha=0.5)
            if not torch.equal(s.index, r.index):
                return None
            return float((host(s.weight) * dw).sum() + host(s.loss)[0])

        h, seen = 2.0**-6, 0
        for t in range(T):
            for e in range(E):
                a, b = l.copy(), l.copy()
                a[t, e] += h
                b[t, e] -= h
                fa, fb = f(a), f(b)
                if fa is None or fb is None:
                    continue
                seen += 1
                assert abs((fa - fb) / (2 * h) - d[t, e]) <= 2e-3
        assert seen > T * E // 2


def test_equal_inputs_equal_bits():
    l = dev(logits(5000, 96, "f32", 2))
    a = bsmm.bsmm_route_topk(l, 6, alpha=1.0)
    for _ in range(3):
        b = bsmm.bsmm_route_topk(l, 6, alpha=1.0)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("T", [5, 500])
def test_streams_and_graph(T):
    l = logits(T, 40, "f32", 6)
    x = dev(l)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    r = bsmm.bsmm_route_topk(x, 4, alpha=1.0, stream=st)
    st.synchronize()
    check_forward(r, R.route(l, 4, alpha=1.0))
    bsmm.bsmm_route_topk(x, 4, alpha=1.0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = bsmm.bsmm_route_topk(x, 4, alpha=1.0)
        d = bsmm.bsmm_route_topk_backward(x, r.index, r.weight, r.counts, r.live,
                                          dloss=torch.ones_like(r.loss), alpha=1.0)
    for i in range(3):
        l2 = logits(T, 40, "f32", 60 + i)
        x.copy_(dev(l2))
        for t in (*r, d):
            t.fill_(-9)
        g.replay()
        torch.cuda.synchronize()
        check_forward(r, R.route(l2, 4, alpha=1.0))
        e = bsmm.bsmm_route_topk_backward(x, r.index, r.weight, r.counts, r.live,
                                          dloss=torch.ones(1, device=DEV), alpha=1.0)
        assert torch.equal(d, e)


def test_overwritten_workspace_stays_in_bounds():
    """Positions that a shared workspace has spoiled are not written past the
    order.  Spoiled here by counts that lie on the first block's row of slots
    before it: that block's slots then move up by their experts' counts."""
    T, E, k = 100, 8, 2
    x = dev(logits(T, E, "f32", 12))
    need = bsmm.bsmm_route_workspace_bytes(T, E)
    blocks = 7                                   # of 16 tokens
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    ints = torch.full((T * k + 1024,), -7, dtype=torch.int32, device=DEV)
    index = torch.empty(T, k, dtype=torch.int32, device=DEV)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    weight = torch.empty(T, k, device=DEV)
    before = ws.data_ptr() + need - blocks * E * 4
    assert bsmm.load().bsmm_route_topk(
        x.data_ptr(), E, bsmm.F32, None, k, 1, 0.0, index.data_ptr(), weight.data_ptr(), before,
        offsets.data_ptr(), ints.data_ptr(), None, None, None, T, E, ws.data_ptr(), need,
        torch.cuda.current_stream().cuda_stream) == 0
    got = host(ints)
    assert (got[T * k:] == -7).all() and (got[:T * k] >= -7).all()
    assert host(offsets)[E] == T * k
    # the last expert's slots of the first block lie behind its run now
    e = host(index).reshape(-1)
    last = np.bincount(e, minlength=E).nonzero()[0][-1]
    hit = np.flatnonzero(e[:16 * k] == last)
    assert hit.size and not np.isin(hit, got[:T * k]).any()
