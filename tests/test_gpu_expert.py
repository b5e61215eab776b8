"""The experts' bf16 and fp32 products and their weight gradient on the GPU.

Checked twice.  On small integers every partial sum is an integer below 2^24,
so any order of fp32 additions is exact and the results must be equal: that
pins indexing, layouts, odd edges and routing.  On normal data the error is
bounded from the sums: n fp32 additions, each off by at most 2^-23 of a partial
sum (truncation), so n 2^-23 sum |a| |b| in all, and an output rounded to bf16
by another 2^-8 of the result, an fp32 one that is scaled by its row by 2^-24.
"""

import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsmm
from oracle import expert as X

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TDT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _lib(gpu_lib):
    yield


def dev(a, dt=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dt is None else t.to(dt)


def host(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def routes(rng, T, E, k, none=0.1, skip=()):
    """(order, offsets) of k choices a token; a share of the slots has no
    expert, and the experts in skip get none."""
    expert = np.stack([rng.permutation([e for e in range(E) if e not in skip] + [E] * k)[:k]
                       for _ in range(T)]).reshape(-1) if T else np.zeros(0, np.int64)
    expert = np.where(rng.random(T * k) < none, E, expert)
    order = np.argsort(expert, kind="stable").astype(np.int32)
    counts = np.bincount(expert, minlength=E + 1)[:E]
    return order, np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def ints(rng, *shape, top=3):
    return rng.integers(-top, top + 1, shape).astype(np.float32)


def strided(a, dt, pad, shift=0):
    """a on the GPU in rows `pad` elements longer, `shift` elements into the
    buffer; NaN around it."""
    R, K = a.shape
    buf = torch.full((R * (K + pad) + shift + pad,), float("nan"), device=DEV).to(dt)
    v = buf[shift:shift + R * (K + pad)].view(R, K + pad)[:, :K]
    v.copy_(dev(a))
    return v


SIZES = [  # T, E, k, N, K
    (1, 3, 1, 64, 64), (1, 8, 2, 1, 1), (2, 4, 2, 16, 7), (5, 4, 3, 33, 31), (7, 7, 3, 129, 65),
    (9, 5, 2, 200, 130), (33, 16, 4, 127, 256), (130, 4, 2, 128, 72), (257, 3, 1, 40, 100),
    (64, 70, 2, 24, 40), (300, 2, 2, 264, 136), (3, 2, 1, 2000, 24), (40, 3, 2, 96, 1000),
]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("T,E,k,N,K", SIZES)
def test_product_exact(T, E, k, N, K, back, dt):
    rng = np.random.default_rng(T * 1000 + N + K)
    order, offsets = routes(rng, T, E, k, skip=(1,) if E > 2 else ())
    w = ints(rng, E, N, K)
    depth = N if back else K
    wg = dev(w, TDT[dt]).transpose(1, 2) if back else dev(w, TDT[dt])
    wh = w.transpose(0, 2, 1) if back else w
    for per in (1, k):
        x = ints(rng, T * k // per, depth)
        scale = np.exp2(rng.integers(-2, 3, T * k)).astype(np.float32)
        for rs in (None, scale):
            got = bsmm.bsmm_expert_mm(dev(x, TDT[dt]), wg, dev(order), dev(offsets),
                                      slots_per_row=per, row_scale=None if rs is None else dev(rs),
                                      out_dtype="f32")
            assert np.array_equal(host(got), X.expert_mm(x, wh, order, offsets, per, rs)), (per, rs)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k,N,K", SIZES)
def test_weight_gradient_exact(T, E, k, N, K, dt):
    rng = np.random.default_rng(T * 1000 + N + K + 1)
    order, offsets = routes(rng, T, E, k, skip=(0,) if E > 2 else ())
    for yper, xper in ((1, k), (k, 1), (1, 1)):
        dy, x = ints(rng, T * k // yper, N), ints(rng, T * k // xper, K)
        got = bsmm.bsmm_expert_wgrad(dev(dy, TDT[dt]), dev(x, TDT[dt]), dev(order), dev(offsets),
                                     dy_slots_per_row=yper, x_slots_per_row=xper)
        assert np.array_equal(host(got), X.expert_wgrad(dy, x, order, offsets, yper, xper))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k,N,K", [(1, 2, 1, 5, 32), (9, 5, 2, 200, 96), (130, 4, 2, 129, 288),
                                       (300, 3, 2, 64, 64)])
def test_weight_gradient_from_checkpoint_exact(T, E, k, N, K, dt):
    rng = np.random.default_rng(T + N)
    order, offsets = routes(rng, T, E, k)
    dy = ints(rng, T * k, N, top=2)
    q = rng.integers(-127, 128, (T, K)).astype(np.int8)
    byte = rng.integers(131, 135, (T, K // 32)).astype(np.uint8)      # steps of 1/4 to 2
    want = X.expert_wgrad(dy, X.restore(q, byte), order, offsets, 1, k)
    assert np.abs(want).max() < 2**21
    got = bsmm.bsmm_expert_wgrad(dev(dy, TDT[dt]), dev(q), dev(order), dev(offsets),
                                 x_scale=dev(byte), x_slots_per_row=k)
    assert np.array_equal(host(got), want)
    # rows at other strides and addresses
    qs = torch.zeros(T, K + 3, dtype=torch.int8, device=DEV)[:, 1:K + 1]
    qs.copy_(dev(q))
    bs = torch.zeros(T, K // 32 + 5, dtype=torch.uint8, device=DEV)[:, 2:K // 32 + 2]
    bs.copy_(dev(byte))
    got = bsmm.bsmm_expert_wgrad(strided(dy, TDT[dt], 3, 1), qs, dev(order), dev(offsets),
                                 x_scale=bs, x_slots_per_row=k, out_dtype="f32")
    assert np.array_equal(host(got), want)


def test_checkpoint_of_nan_gives_nan():
    """Byte 255 in one block of one row: its expert's columns, and no other."""
    dy = torch.ones(4, 8, device=DEV, dtype=torch.bfloat16)
    q = torch.ones(4, 96, device=DEV, dtype=torch.int8)
    byte = torch.full((4, 3), 133, device=DEV, dtype=torch.uint8)
    byte[2, 1] = 255
    got = host(bsmm.bsmm_expert_wgrad(dy, q, None, dev(np.array([0, 2, 4], np.int32)),
                                      x_scale=byte))
    assert np.isnan(got[1, :, 32:64]).all()
    got[1, :, 32:64] = 2.0
    assert (got == 2.0).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (3, 1), (0, 3), (4, 8)])
def test_strides(dt, pad, shift):
    """Rows longer than their contents and unaligned, NaN around the operands
    and a guard around the output."""
    rng = np.random.default_rng(7)
    T, E, k, N, K = 50, 3, 2, 70, 90
    order, offsets = routes(rng, T, E, k)
    x, w = ints(rng, T, K), ints(rng, E, N, K)
    want = X.expert_mm(x, w, order, offsets, k)
    wide = strided(w.reshape(E * N, K), TDT[dt], pad, shift).unflatten(0, (E, N))
    out = torch.full((T * k + 2, N + 5), 99.0, device=DEV)
    bsmm.bsmm_expert_mm(strided(x, TDT[dt], pad, shift), wide, dev(order), dev(offsets),
                        slots_per_row=k, out_dtype="f32", out=out[1:-1, 2:N + 2])
    got = host(out)
    assert np.array_equal(got[1:-1, 2:N + 2], want)
    got[1:-1, 2:N + 2] = 99.0
    assert (got == 99.0).all()

    dy = ints(rng, T * k, N)
    dx = bsmm.bsmm_expert_mm(strided(dy, TDT[dt], pad, shift), wide.transpose(1, 2), dev(order),
                             dev(offsets), out_dtype="f32")
    assert np.array_equal(host(dx), X.expert_mm(dy, w.transpose(0, 2, 1), order, offsets))

    dw = torch.full((E, N + 2, K + 3), 99.0, device=DEV)
    bsmm.bsmm_expert_wgrad(strided(dy, TDT[dt], pad, shift), strided(x, TDT[dt], pad, shift),
                           dev(order), dev(offsets), x_slots_per_row=k, out=dw[:, 1:N + 1, 1:K + 1])
    got = host(dw)
    assert np.array_equal(got[:, 1:N + 1, 1:K + 1], X.expert_wgrad(dy, x, order, offsets, 1, k))
    got[:, 1:N + 1, 1:K + 1] = 99.0
    assert (got == 99.0).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_sorted_slots_without_order(dt):
    """order None: a dense layer with one expert, and sorted rows with more;
    rows behind the last expert are zeros."""
    rng = np.random.default_rng(8)
    x, w, dy = ints(rng, 200, 48), ints(rng, 3, 40, 48), ints(rng, 200, 40)
    for offsets in ([0, 200, 200, 200], [0, 1, 150, 190], [0, 0, 0, 0]):
        off = np.array(offsets, np.int32)
        got = bsmm.bsmm_expert_mm(dev(x, TDT[dt]), dev(w, TDT[dt]), None, dev(off), out_dtype="f32")
        assert np.array_equal(host(got), X.expert_mm(x, w, None, off))
        got = bsmm.bsmm_expert_wgrad(dev(dy, TDT[dt]), dev(x, TDT[dt]), None, dev(off))
        assert np.array_equal(host(got), X.expert_wgrad(dy, x, None, off))
    # each of 100 rows twice
    got = bsmm.bsmm_expert_mm(dev(x[:100], TDT[dt]), dev(w, TDT[dt]), None, dev(off := np.array(
        [0, 60, 61, 200], np.int32)), slots_per_row=2, out_dtype="f32")
    assert np.array_equal(host(got), X.expert_mm(x[:100], w, None, off, 2))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("odt", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k,N,K", [(1, 8, 4, 512, 1024), (12, 8, 2, 513, 1031),
                                       (300, 4, 2, 384, 2048), (700, 2, 1, 260, 520)])
def test_accuracy(T, E, k, N, K, dt, odt):
    rng = np.random.default_rng(N)
    order, offsets = routes(rng, T, E, k, none=0.0)
    g = TDT[dt]
    x, w = dev(rng.standard_normal((T, K)), g), dev(rng.standard_normal((E, N, K)), g)
    dy, r = dev(rng.standard_normal((T * k, N)), g), rng.random(T * k).astype(np.float32)
    xh, wh, dyh = host(x), host(w), host(dy)
    last = 2.0**-8 if odt == "bf16" else 2.0**-24

    def check(got, want, size, n):
        assert got.dtype == TDT[odt]
        limit = n * 2.0**-23 * size + (last + 2.0**-23) * np.abs(want)
        assert (np.abs(host(got) - want) <= limit).all()

    def mm(a, b, **kw):
        return X.expert_mm(a, b, order, offsets, **kw)

    got = bsmm.bsmm_expert_mm(x, w, dev(order), dev(offsets), slots_per_row=k, row_scale=dev(r),
                              out_dtype=odt)
    check(got, mm(xh, wh, slots_per_row=k, row_scale=r),
          mm(np.abs(xh), np.abs(wh), slots_per_row=k, row_scale=r), K)
    wt = wh.transpose(0, 2, 1)
    got = bsmm.bsmm_expert_mm(dy, w.transpose(1, 2), dev(order), dev(offsets), out_dtype=odt)
    check(got, mm(dyh, wt), mm(np.abs(dyh), np.abs(wt)), N)
    got = bsmm.bsmm_expert_wgrad(dy, x, dev(order), dev(offsets), x_slots_per_row=k, out_dtype=odt)
    check(got, X.expert_wgrad(dyh, xh, order, offsets, 1, k),
          X.expert_wgrad(np.abs(dyh), np.abs(xh), order, offsets, 1, k),
          int(np.diff(offsets).max()))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_keep_to_themselves(dt):
    """A NaN in one row reaches its own slots (and its experts' gradients)
    only, an infinite weight its own expert only, and equal calls give equal
    bits."""
    rng = np.random.default_rng(9)
    T, E, k, N, K = 90, 4, 2, 100, 200
    order, offsets = routes(rng, T, E, k)
    x, w = rng.standard_normal((T, K)), rng.standard_normal((E, N, K))
    args = dev(order), dev(offsets)
    clean = host(bsmm.bsmm_expert_mm(dev(x, TDT[dt]), dev(w, TDT[dt]), *args, slots_per_row=k))
    x[17, 5] = np.nan
    w[2, 3, 7] = np.inf
    got = host(bsmm.bsmm_expert_mm(dev(x, TDT[dt]), dev(w, TDT[dt]), *args, slots_per_row=k))
    again = host(bsmm.bsmm_expert_mm(dev(x, TDT[dt]), dev(w, TDT[dt]), *args, slots_per_row=k))
    assert np.array_equal(got, again, equal_nan=True)
    mine = np.zeros((T * k, N), bool)
    used = set(order[:offsets[E]])
    for s in (34, 35):
        mine[s] = s in used
    mine[order[offsets[2]:offsets[3]], 3] = True
    assert not np.isfinite(got[mine]).any()
    assert np.array_equal(got[~mine], clean[~mine])

    dy = rng.standard_normal((T * k, N))
    with np.errstate(invalid="ignore"):
        x0 = np.where(np.isnan(x), 0.0, x)
    clean = host(bsmm.bsmm_expert_wgrad(dev(dy, TDT[dt]), dev(x0, TDT[dt]), *args, x_slots_per_row=k))
    got = host(bsmm.bsmm_expert_wgrad(dev(dy, TDT[dt]), dev(x, TDT[dt]), *args, x_slots_per_row=k))
    reach = np.zeros_like(got, dtype=bool)
    for e in range(E):
        if {34, 35} & set(order[offsets[e]:offsets[e + 1]]):
            reach[e, :, 5] = True
    assert np.isnan(got[reach]).all() and np.array_equal(got[~reach], clean[~reach])


def test_empty_sizes():
    i = torch.int32
    z = torch.zeros
    off = z(3, dtype=i, device=DEV)
    none = z(0, dtype=i, device=DEV)
    assert bsmm.bsmm_expert_mm(z(0, 8, device=DEV), z(2, 4, 8, device=DEV), none, off).shape == (0, 4)
    assert bsmm.bsmm_expert_mm(z(3, 8, device=DEV), z(2, 0, 8, device=DEV), None, off).shape == (3, 0)
    got = bsmm.bsmm_expert_mm(z(3, 0, device=DEV), z(2, 4, 0, device=DEV), None,
                              dev(np.array([0, 2, 3], np.int32)),
                              out=torch.ones(3, 4, device=DEV, dtype=torch.bfloat16))
    assert got.shape == (3, 4) and not host(got).any()
    got = bsmm.bsmm_expert_wgrad(z(0, 5, device=DEV), z(0, 8, device=DEV), none, off,
                                 out=torch.ones(2, 5, 8, device=DEV))
    assert not host(got).any()


def test_other_stream_and_graph():
    """On a stream of its own, and captured and replayed on changed inputs."""
    rng = np.random.default_rng(10)
    T, E, k, N, K = 60, 5, 2, 136, 264
    x, w = dev(ints(rng, T, K), torch.bfloat16), dev(ints(rng, E, N, K), torch.bfloat16)
    order, offsets = (dev(a) for a in routes(rng, T, E, k))

    def both():
        y = bsmm.bsmm_expert_mm(x, w, order, offsets, slots_per_row=k)
        return y, bsmm.bsmm_expert_wgrad(y, x, order, offsets, x_slots_per_row=k)

    want = [host(t) for t in both()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = both()
    s.synchronize()
    assert all(np.array_equal(host(a), b) for a, b in zip(got, want))
    y = bsmm.bsmm_expert_mm(x, w, order, offsets, slots_per_row=k, stream=s)
    s.synchronize()
    assert np.array_equal(host(y), want[0])

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        static = both()
    for i in range(4):
        x.copy_(dev(ints(rng, T, K)))
        o, f = routes(rng, T, E, k, none=0.2 * i)
        order.copy_(dev(o))
        offsets.copy_(dev(f))
        graph.replay()
        torch.cuda.synchronize()
        got = [host(t) for t in static]
        assert all(np.array_equal(a, host(b)) for a, b in zip(got, both())), i
