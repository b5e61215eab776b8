"""Calls that need a workspace, in graphs and from several threads: a graph's
memory is its own, whatever eager calls or other graphs do between its
replays, and so is a host thread's.  Integers as in
the products' tests, so that results must be equal."""

import threading

import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsmm
from oracle import route as R, w4
from synth import fp8_mx_bmm_inputs, int8_rowwise_inputs
from test_gpu_route import check_forward, logits
from test_gpu_w4 import dev, integer_case, same

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _lib(gpu_lib):
    yield


class RouteCall:
    """The router on T tokens: three launches through a workspace."""

    def __init__(self, T, E=40, k=4):
        self.T, self.E, self.k = T, E, k
        self.need = bsmm.bsmm_route_workspace_bytes(T, E)
        self.x = torch.empty(T, E, device=DEV)

    def feed(self, seed):
        self.host = logits(self.T, self.E, "f32", seed)
        self.x.copy_(dev(self.host))

    def run(self, **kw):
        self.out = bsmm.bsmm_route_topk(self.x, self.k, alpha=1.0, **kw)

    def clear(self):
        for t in self.out:
            t.fill_(-9)

    def check(self):
        check_forward(self.out, R.route(self.host, self.k, alpha=1.0))


class ProductCall:
    """fp32 activations on tiles: two launches through a workspace."""

    def __init__(self, M, N=2100, K=512):
        self.M, self.N, self.K = M, N, K
        self.need = bsmm.bsmm_w4_workspace_bytes("f32", 1, M, M, N, K, 64)
        c = integer_case(M, N, K, 64, True, "f32", 3)
        self.w = [c["q"], c["s"], c["z"]]
        self.dw = [dev(t) for t in self.w]
        self.x = torch.empty(M, K, device=DEV)

    def feed(self, seed):
        self.host = np.random.default_rng(seed).integers(-3, 4, (self.M, self.K)) \
            .astype(np.float32)
        self.x.copy_(dev(self.host))

    def run(self, **kw):
        self.out = bsmm.bsmm_w4_mm(self.x, *self.dw, out_dtype="f32", **kw)

    def clear(self):
        self.out.fill_(-9)

    def check(self):
        same(self.out, w4.w4_mm(self.host, *self.w), "f32")


CALLS = [(RouteCall, 300, 6000), (ProductCall, 1300, 2048)]


def captured(call, **kw):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, **kw):
        call.run()
    return g


@pytest.mark.parametrize("kind,size,larger", CALLS)
def test_graph_after_a_larger_eager_call(kind, size, larger):
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call = kind(size)
        assert call.need > 0
        call.feed(0)
        call.run()
        g = captured(call, stream=s)
        big = kind(larger)
        assert big.need > call.need
        big.feed(1)
        big.run()
        others = [torch.full((call.need,), 0x5A, dtype=torch.uint8, device=DEV) for _ in range(8)]
        for i in range(3):
            call.feed(10 + i)
            call.clear()
            big.run()
            g.replay()
            s.synchronize()
            call.check()
            big.check()
            assert all((t == 0x5A).all() for t in others)


@pytest.mark.parametrize("kind,size,_", CALLS)
def test_two_graphs_at_once(kind, size, _):
    calls = [kind(size), kind(size)]
    for i, c in enumerate(calls):
        c.feed(20 + i)
        c.run()
    torch.cuda.synchronize()
    graphs = [captured(c) for c in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(3):
        for j, c in enumerate(calls):
            c.feed(30 + 2 * i + j)
            c.clear()
        torch.cuda.synchronize()
        for _ in range(4):
            for s, g in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for c in calls:
            c.check()


@pytest.mark.parametrize("kind,size,larger", CALLS)
def test_threads_on_one_stream(kind, size, larger):
    s = torch.cuda.Stream()
    calls = [kind(size), kind(larger), kind(size)]
    for i, c in enumerate(calls):
        c.feed(40 + i)
    torch.cuda.synchronize()
    start, errors = threading.Barrier(len(calls)), []

    def work(c):
        try:
            start.wait(30)
            with torch.cuda.stream(s):
                for _ in range(20):
                    c.run()
                s.synchronize()
        except Exception as e:      # reported by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not errors
    for c in calls:
        c.check()


@pytest.mark.parametrize("kind,size,_", CALLS)
def test_given_workspace(kind, size, _):
    """The caller's buffer is the one that is used, and no byte past it."""
    call = kind(size)
    call.feed(50)
    buf = torch.full((call.need + 256,), 0x5A, dtype=torch.uint8, device=DEV)
    cached = dict(bsmm._WS.by)
    call.run(workspace=buf[:call.need])
    call.check()
    assert bsmm._WS.by == cached
    assert not (buf[:call.need] == 0x5A).all() and (buf[call.need:] == 0x5A).all()


def test_product_without_workspace():
    call = ProductCall(300)
    call.feed(51)
    for ws in (False, torch.empty(16, dtype=torch.uint8, device=DEV)):
        call.run(workspace=ws)
        call.check()


def gemm(kind):
    """(a call whose tiles are split between workgroups, counted in the
    workspace; the operand to change between calls; other contents for it)"""
    if kind == "narrow":
        G, M, N, K = 8, 128, 1024, 4096
        plan = bsmm.bsmm_query_plan(bsmm.OP_FP8_MX_BMM, G, M, N, K, "bf16")
        assert plan["variant"].startswith("n128") and plan["split_k"] > 1, plan
        ps = [fp8_mx_bmm_inputs(G, M, N, K, i) for i in range(3)]
        x, w, sx, sw = (dev(ps[0][n]) for n in ("x", "w", "x_scale", "w_scale"))
        return (lambda **kw: bsmm.bsmm_fp8_mx_bmm(x, w, sx, sw, layout=ps[0]["layout"], **kw),
                x, [dev(p["x"]) for p in ps])
    M, N, K = 2048, 2304, 512
    bsmm.bsmm_set_override("t256x256skp", 0)
    ps = [int8_rowwise_inputs(M, N, K, i) for i in range(3)]
    a, b = dev(ps[0]["a"]), dev(ps[0]["b_nk"]).t()
    sa, sb = dev(ps[0]["scale_a"]).reshape(-1, 1), dev(ps[0]["scale_b"]).reshape(1, -1)
    return (lambda **kw: bsmm.bsmm_int8_rowwise(a, b, sa, sb, **kw), a,
            [dev(p["a"]) for p in ps])


@pytest.mark.parametrize("kind", ["narrow", "stream-K"])
def test_graph_of_a_split_gemm(kind):
    """Every replay counts its tiles' parts anew: the counters hold a tag of
    the launch, which replays share."""
    try:
        if kind == "stream-K":
            bsmm.bsmm_set_streamk_grid(50)
        call, operand, contents = gemm(kind)
        want = []
        for t in contents:
            operand.copy_(t)
            want.append(call().clone())
        out = torch.empty_like(want[0])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(out=out)
        for i in (0, 1, 2, 0, 1):
            operand.copy_(contents[i])
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[i]), i
    finally:
        bsmm.bsmm_set_override(None, 0)
        bsmm.bsmm_set_streamk_grid(0)
