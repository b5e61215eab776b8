"""The kernels of the experts' products where they hand over to each other:
items of every height, few rows, odd sizes, sums over parts of the
contraction, rows further apart than 32 bits reach.  Small integers, so that
every order of fp32 additions is exact (see test_gpu_expert.py)."""

import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsmm
from oracle import expert as X
from test_gpu_expert import DEV, TDT, dev, host, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(gpu_lib):
    yield


def sorted_offsets(loads):
    return np.concatenate([[0], np.cumsum(loads)]).astype(np.int32)


# loads of the experts: every number of 64-row blocks, full items and one row more
LOADS = [
    [1, 63, 64, 65, 128, 129, 192, 193, 256, 257, 0, 300, 511, 512, 513],
    [700, 0, 3], [255, 1], [16] * 20, [17] * 20, [90] * 12,
]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("loads", LOADS, ids=lambda v: f"{len(v)}x{max(v)}")
def test_item_heights(loads, back, dt):
    rng = np.random.default_rng(sum(loads))
    off, S, E = sorted_offsets(loads), sum(loads) + 5, len(loads)      # 5 slots without an expert
    for N, K in ((264, 72), (40, 328), (520, 8), (320, 640)):
        w = ints(rng, E, N, K, top=2)
        x = ints(rng, S, N if back else K, top=2)
        wg, wh = (dev(w, TDT[dt]).transpose(1, 2), w.transpose(0, 2, 1)) if back else \
            (dev(w, TDT[dt]), w)
        order = rng.permutation(S).astype(np.int32)
        for o in (None, order):
            got = bsmm.bsmm_expert_mm(dev(x, TDT[dt]), wg, None if o is None else dev(o), dev(off),
                                      out_dtype="f32")
            assert np.array_equal(host(got), X.expert_mm(x, wh, o, off)), (N, K, o is None)
        got = bsmm.bsmm_expert_mm(dev(x, TDT[dt]), wg, dev(order), dev(off))
        want = torch.from_numpy(X.expert_mm(x, wh, order, off)).to(torch.bfloat16)
        assert np.array_equal(host(got), want.double().numpy())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("loads", LOADS, ids=lambda v: f"{len(v)}x{max(v)}")
def test_gradient_runs(loads, dt):
    rng = np.random.default_rng(sum(loads) + 1)
    off, S = sorted_offsets(loads), sum(loads) + 5
    order = rng.permutation(S).astype(np.int32)
    for N, K in ((264, 72), (4, 260), (300, 516), (33, 31)):
        dy, x = ints(rng, S, N, top=2), ints(rng, S, K, top=2)
        want = X.expert_wgrad(dy, x, order, off)
        got = bsmm.bsmm_expert_wgrad(dev(dy, TDT[dt]), dev(x, TDT[dt]), dev(order), dev(off))
        assert np.array_equal(host(got), want), (N, K)
        got = bsmm.bsmm_expert_wgrad(dev(dy, TDT[dt]), dev(x, TDT[dt]), dev(order), dev(off),
                                     out_dtype="bf16")
        assert np.array_equal(host(got), torch.from_numpy(want).to(torch.bfloat16).double().numpy())


# on average 16 rows or fewer, with items of one block of 16, of two, and second items
FEW = [[0, 1, 15, 16, 17, 31, 32, 33, 64, 5, 0, 2, 20, 3, 1, 0], [1] * 16, [20, 12] * 8]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("N,K", [(1030, 40), (1024, 1032), (4100, 8), (200, 520)])
@pytest.mark.parametrize("loads", FEW, ids=lambda v: f"{len(v)}x{max(v)}")
def test_few_rows(loads, N, K, back, dt):
    rng = np.random.default_rng(sum(loads) + N)
    if back:
        N, K = K, N // 8 * 8                              # [E, K, N] in memory, rows of 8
    off, S, E = sorted_offsets(loads), sum(loads) + 5, len(loads)
    x, w = ints(rng, S, K, top=2), ints(rng, E, N, K, top=2)
    wg = dev(w.transpose(0, 2, 1).copy(), TDT[dt]).transpose(1, 2) if back else dev(w, TDT[dt])
    order = rng.permutation(S).astype(np.int32)
    scale = np.exp2(rng.integers(-2, 3, S)).astype(np.float32)
    got = bsmm.bsmm_expert_mm(dev(x, TDT[dt]), wg, dev(order), dev(off), row_scale=dev(scale),
                              out_dtype="f32")
    assert np.array_equal(host(got), X.expert_mm(x, w, order, off, 1, scale))


ODD = [(261, 333), (258, 129), (1031, 67), (515, 640), (7, 70), (4, 1), (3, 65), (256, 250),
       (513, 15)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("N,K", ODD)
def test_odd_sizes(N, K, shift, dt):
    """Rows that end in a unit, tiles that end in four columns, and rows that
    begin at any element; what surrounds the rows is NaN."""
    rng = np.random.default_rng(N * K + shift)
    t, loads = TDT[dt], LOADS[0]
    off, S, E = sorted_offsets(loads), sum(loads) + 5, len(loads)
    order = rng.permutation(S).astype(np.int32)

    def inside(v):
        """v as a view into a wider tensor of NaN."""
        wide = torch.full((*v.shape[:-1], v.shape[-1] + shift + 2), float("nan"), device=DEV,
                          dtype=t)
        wide[..., shift:shift + v.shape[-1]] = dev(v, t)
        return wide[..., shift:shift + v.shape[-1]]

    x, w, y = ints(rng, S, K, top=2), ints(rng, E, N, K, top=2), ints(rng, S, N, top=2)
    xg, yg, og, fg = inside(x), inside(y), dev(order), dev(off)
    got = bsmm.bsmm_expert_mm(xg, inside(w), og, fg, out_dtype="f32")
    assert np.array_equal(host(got), X.expert_mm(x, w, order, off))
    wt = inside(w.transpose(0, 2, 1)).transpose(1, 2)                     # contiguous along N
    for odt in ("f32", "bf16"):
        o = inside(np.zeros((S, N))) if odt == dt else None
        got = bsmm.bsmm_expert_mm(xg, wt, og, fg, out_dtype=odt, out=o)
        want = torch.from_numpy(X.expert_mm(x, w, order, off)).to(TDT[odt]).double().numpy()
        assert np.array_equal(host(got), want), odt
        if o is not None:
            rest = o._base.clone()
            rest[..., shift:shift + N] = float("nan")
            assert rest.isnan().all()
        o = inside(np.zeros((E, N, K))) if odt == dt else None
        got = bsmm.bsmm_expert_wgrad(yg, xg, og, fg, out_dtype=odt, out=o)
        want = torch.from_numpy(X.expert_wgrad(y, x, order, off)).to(TDT[odt]).double().numpy()
        assert np.array_equal(host(got), want), odt
        if o is not None:
            rest = o._base.clone()
            rest[..., shift:shift + K] = float("nan")
            assert rest.isnan().all()


PARTS = [  # few tiles and a long contraction
    ("mm", 300, 2, 130, 4096), ("mm", 300, 2, 130, 4099), ("mm", 70, 1, 64, 9000),
    ("wgrad", 9000, 1, 64, 72), ("wgrad", 9000, 2, 33, 31), ("wgrad", 20000, 1, 256, 512),
]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("op,S,E,N,K", PARTS)
def test_parts(op, S, E, N, K, dt):
    """With a workspace of its own (filled with NaN), with none, and with one
    that is too small: the same result."""
    rng = np.random.default_rng(S + N)
    off = sorted_offsets([S // E - 1] * E)
    order = rng.permutation(S).astype(np.int32)
    scale = np.exp2(rng.integers(-2, 3, S)).astype(np.float32)
    code = bsmm.BF16 if dt == "bf16" else bsmm.F32
    if op == "mm":
        x, w = ints(rng, S, K, top=1), ints(rng, E, N, K, top=1)
        need = bsmm.bsmm_expert_mm_workspace_bytes(code, False, E, S, N, K)
        want = X.expert_mm(x, w, order, off, 1, scale)
        call = lambda ws: bsmm.bsmm_expert_mm(  # noqa: E731
            dev(x, TDT[dt]), dev(w, TDT[dt]), dev(order), dev(off), row_scale=dev(scale),
            out_dtype="f32", workspace=ws)
    else:
        dy, x = ints(rng, S, N, top=1), ints(rng, S, K, top=1)
        need = bsmm.bsmm_expert_wgrad_workspace_bytes(code, False, E, S, S, N, K)
        want = X.expert_wgrad(dy, x, order, off)
        call = lambda ws: bsmm.bsmm_expert_wgrad(  # noqa: E731
            dev(dy, TDT[dt]), dev(x, TDT[dt]), dev(order), dev(off), workspace=ws)
    assert need > 0
    nan = torch.full((need // 4 + 4,), float("nan"), device=DEV)
    for ws in (None, False, nan, nan[:need // 8]):
        assert np.array_equal(host(call(ws)), want)


@pytest.mark.parametrize("odt", ["bf16", "f32"])
def test_checkpoint_workspace(odt):
    """The codes restored first (wide tiles), or read as they are."""
    rng = np.random.default_rng(3)
    off, order = sorted_offsets([300, 0, 451, 80]), rng.permutation(840).astype(np.int32)
    dy, N, K = ints(rng, 840, 512, top=1), 512, 320
    q = rng.integers(-9, 10, (420, K)).astype(np.int8)
    byte = rng.integers(131, 134, (420, K // 32)).astype(np.uint8)
    want = X.expert_wgrad(dy, X.restore(q, byte), order, off, 1, 2)
    if odt == "bf16":
        want = torch.from_numpy(want).to(torch.bfloat16).double().numpy()
    need = bsmm.bsmm_expert_wgrad_workspace_bytes("bf16", True, 4, 420, 840, N, K)
    assert need >= 420 * K * 2
    nan = torch.full((need // 4 + 4,), float("nan"), device=DEV)
    for ws in (None, False, nan):
        got = bsmm.bsmm_expert_wgrad(dev(dy, torch.bfloat16), dev(q), dev(order), dev(off),
                                     x_scale=dev(byte), x_slots_per_row=2, out_dtype=odt,
                                     workspace=ws)
        assert np.array_equal(host(got), want)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("codes", [False, True])
def test_gradient_of_many_tiles(codes, dt):
    """Long runs and many columns, without a workspace."""
    rng = np.random.default_rng(9)
    S, N, K, t = 2000, 2047, 2048, TDT[dt]
    off, order = sorted_offsets([900, 1090]), rng.permutation(S).astype(np.int32)
    dy, x = ints(rng, S, N, top=1), ints(rng, S, K, top=1)
    scale = np.full((S, K // 32), 133, np.uint8)
    xg = dev(x.astype(np.int8)) if codes else dev(x, t)
    got = bsmm.bsmm_expert_wgrad(dev(dy, t), xg, dev(order), dev(off), workspace=False,
                                 x_scale=dev(scale) if codes else None)
    assert np.array_equal(host(got), X.expert_wgrad(dy, x, order, off))


def far(shape, row, dt):
    """[rows, cols] whose rows are `row` elements apart, zeros."""
    buf = torch.empty(row * (shape[0] - 1) + shape[1], device=DEV, dtype=dt)
    v = buf.as_strided(shape, (row, 1))
    v.zero_()
    return v


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_far_apart(dt):
    """Row strides past 2^31 bytes and elements: the operands', the outputs'
    and the experts'."""
    rng = np.random.default_rng(4)
    t, row = TDT[dt], 2**31 // 2 + 64
    S, N, K, E = 3, 64, 72, 3
    off = sorted_offsets([1, 1, 1])
    xh, wh, dyh = ints(rng, S, K), ints(rng, E, N, K), ints(rng, S, N)
    x, out = far((S, K), row, t), far((S, N), row, torch.float32)
    x.copy_(dev(xh))
    w = far((E, N * K), row, t).unflatten(1, (N, K))
    w.copy_(dev(wh))
    got = bsmm.bsmm_expert_mm(x, w, None, dev(off), out=out, out_dtype="f32")
    assert np.array_equal(host(got), X.expert_mm(xh, wh, None, off))
    dw = far((E, N * K), row, torch.float32).unflatten(1, (N, K))
    dy = far((S, N), row, t)
    dy.copy_(dev(dyh))
    got = bsmm.bsmm_expert_wgrad(dy, x, None, dev(off), out=dw)
    assert np.array_equal(host(got), X.expert_wgrad(dyh, xh, None, off))
    del got, dw, w, out
    # many rows to an expert: the tiles
    off = sorted_offsets([3])
    w1 = dev(wh[:1], t)
    got = bsmm.bsmm_expert_mm(dy, w1.transpose(1, 2), None, dev(off), out_dtype="f32")
    assert np.array_equal(host(got), X.expert_mm(dyh, wh[:1].transpose(0, 2, 1), None, off))


def test_weights_beyond_two_gigabytes():
    """The last of 20 experts of 8192 x 8192 (2.7 GB of bf16)."""
    E, N, K, rows = 20, 8192, 8192, 70
    w = torch.zeros(E, N, K, device=DEV, dtype=torch.bfloat16)
    w[E - 1, 5, 9], w[E - 1, N - 1, K - 1] = 2.0, 3.0
    x = torch.ones(rows, K, device=DEV, dtype=torch.bfloat16)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[E] = rows
    y = host(bsmm.bsmm_expert_mm(x, w, None, off, out_dtype="f32"))
    assert (y[:, 5] == 2).all() and (y[:, N - 1] == 3).all() and y.sum() == 5 * rows
    dx = host(bsmm.bsmm_expert_mm(x, w.transpose(1, 2), None, off, out_dtype="f32"))
    assert (dx[:, 9] == 2).all() and (dx[:, K - 1] == 3).all() and dx.sum() == 5 * rows
    dw = bsmm.bsmm_expert_wgrad(x, x, None, off, out_dtype="bf16")
    assert not dw[:E - 1].any() and (dw[E - 1] == rows).all()


def test_contents_of_order_and_offsets_stay_inside():
    """Slots and offsets that no router writes give some result and touch
    nothing else: a guard around every output."""
    rng = np.random.default_rng(6)
    S, E, N, K = 150, 4, 72, 64
    x, w = dev(ints(rng, S, K), torch.bfloat16), dev(ints(rng, E, N, K), torch.bfloat16)
    dy = dev(ints(rng, S, N), torch.bfloat16)
    out = torch.full((S + 2, N), 7.0, device=DEV)
    dw = torch.full((E + 2, N, K), 7.0, device=DEV)
    for order in (rng.integers(-2**31, 2**31, S), rng.integers(-3, S + 3, S), np.zeros(S)):
        for off in ([0, 50, 20, 90, 150], [5, -7, 2**31 - 1, 3, 2**31 - 1], [150, 0, 150, 0, 150]):
            o, f = dev(order.astype(np.int32)), dev(np.array(off, np.int64).astype(np.int32))
            bsmm.bsmm_expert_mm(x, w, o, f, out=out[1:-1], out_dtype="f32")
            bsmm.bsmm_expert_wgrad(dy, x, o, f, out=dw[1:-1])
    torch.cuda.synchronize()
    assert (out[0] == 7).all() and (out[-1] == 7).all()
    assert (dw[0] == 7).all() and (dw[-1] == 7).all()


def test_two_threads_on_one_stream():
    """Calls of several launches from two host threads, each with its own
    workspace."""
    import threading
    rng = np.random.default_rng(7)
    S, N, K = 9000, 64, 72
    off = dev(sorted_offsets([S]))
    data = [(dev(ints(rng, S, N, top=1), torch.bfloat16), dev(ints(rng, S, K, top=1),
                                                             torch.bfloat16)) for _ in range(2)]
    want = [host(bsmm.bsmm_expert_wgrad(a, b, None, off, workspace=False)) for a, b in data]
    bad = []

    def work(i):
        for _ in range(20):
            got = bsmm.bsmm_expert_wgrad(*data[i], None, off)
            if not np.array_equal(host(got), want[i]):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_two_graphs_share_nothing():
    """Two captured calls that want a workspace, replayed on two streams at a
    time between eager calls of other sizes."""
    rng = np.random.default_rng(8)
    S, N, K = 9000, 64, 72
    off = dev(sorted_offsets([S]))
    data = [(dev(ints(rng, S, N, top=1), torch.bfloat16), dev(ints(rng, S, K, top=1),
                                                             torch.bfloat16)) for _ in range(2)]
    want = [host(bsmm.bsmm_expert_wgrad(a, b, None, off)) for a, b in data]
    graphs, outs = [], []
    torch.cuda.synchronize()
    for a, b in data:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(bsmm.bsmm_expert_wgrad(a, b, None, off))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    big = dev(ints(rng, 20000, 256, top=1), torch.bfloat16)
    for _ in range(4):
        for o in outs:
            o.fill_(99.0)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        bsmm.bsmm_expert_wgrad(big, big, None, dev(sorted_offsets([20000])))
        torch.cuda.synchronize()
        assert all(np.array_equal(host(o), w) for o, w in zip(outs, want))
