"""The kernels of the experts' products and their weight gradient, each named
and checked to be the one that the sizes take: rows of any alignment in the
wide tiles, items of every height, restored checkpoints, rows, columns and
experts further apart than 32 bits reach.  Small integers, so that every order
of fp32 additions is exact (see test_gpu_expert.py)."""

import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsmm
from oracle import expert as X
from test_gpu_expert import DEV, TDT, dev, host, ints
from test_gpu_expert_paths import far, sorted_offsets

pytestmark = pytest.mark.gpu

mm_name, wgrad_name = bsmm.bsmm_expert_mm_plan_name, bsmm.bsmm_expert_wgrad_plan_name


@pytest.fixture(autouse=True)
def _lib(gpu_lib):
    yield


def product(x, w, order, off, per=1):
    """X.expert_mm, an expert at a time."""
    x, w = x.astype(np.float64), w.astype(np.float64)
    S = len(x) * per if order is None else len(order)
    out = np.zeros((S, w.shape[1]))
    for e in range(len(w)):
        s = X.slots_of(order, off, e, S)
        out[s] = x[s // per] @ w[e].T
    return out


def as_type(want, dt):
    return torch.from_numpy(want).to(TDT[dt]).double().numpy()


def inside(v, dt, shift, after=2, fill=float("nan")):
    """v as a view into a wider tensor of NaN."""
    wide = torch.full((*v.shape[:-1], v.shape[-1] + shift + after), fill, device=DEV, dtype=TDT[dt])
    wide[..., shift:shift + v.shape[-1]] = dev(v, TDT[dt])
    return wide[..., shift:shift + v.shape[-1]]


def only_inside(o, shift):
    """Whether what surrounds such a view is still NaN."""
    rest = o._base.clone()
    rest[..., shift:shift + o.shape[-1]] = float("nan")
    return bool(rest.isnan().all())


# loads with experts without rows, of every number of 64-row blocks, and many rows
RAGGED = [700, 0, 1025, 300, 5, 64, 129, 450]
EVEN = [333] * 8 + [100, 0, 257, 31]
MANY = [1500, 1025, 0, 1200, 1111, 980, 1300, 1023, 1]

# every remainder of N and K by 4 and of K by 8
ODD = [(RAGGED, 1001, 2051, "wide128"), (RAGGED, 1002, 1043, "wide128"),
       (RAGGED, 1003, 1030, "wide128"), (RAGGED, 1031, 517, "wide128"),
       (EVEN, 2049, 515, "wide192"), (EVEN, 770, 2052, "wide128"), (RAGGED, 2048, 2001, "wide128"),
       (MANY, 2050, 1025, "wide256"), (MANY, 2049, 518, "wide256"), (MANY, 1001, 1300, "wide192")]


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("loads,N,K,name", ODD, ids=lambda v: str(v) if isinstance(v, int) else "")
def test_wide_tiles_of_any_alignment(loads, N, K, name, shift):
    """Rows that begin anywhere and end inside a unit or four columns, with
    what surrounds them NaN, in both directions and the gradient."""
    rng = np.random.default_rng(N * K + shift)
    off, S, E = sorted_offsets(loads), sum(loads) + 5, len(loads)     # 5 slots without an expert
    order = rng.permutation(S).astype(np.int32)
    og, fg = dev(order), dev(off)
    assert mm_name("bf16", False, E, S, N, K, aligned=False) == (name, 1)
    x, w = ints(rng, S, K, top=2), ints(rng, E, N, K, top=2)
    xg = inside(x, "bf16", shift)
    want = product(x, w, order, off)
    for along in (True, False):
        wg = inside(w, "bf16", shift) if along else \
            inside(w.transpose(0, 2, 1), "bf16", shift).transpose(1, 2)
        for odt in ("f32", "bf16"):
            o = inside(np.zeros((S, N)), odt, shift)
            got = bsmm.bsmm_expert_mm(xg, wg, og, fg, out_dtype=odt, out=o)
            assert np.array_equal(host(got), as_type(want, odt)), (along, odt)
            assert only_inside(o, shift)
    dy = ints(rng, S, N, top=2)
    want = np.zeros((E, N, K))
    for e in range(E):
        s = order[off[e]:off[e + 1]]
        want[e] = dy[s].astype(np.float64).T @ x[s].astype(np.float64)
    for odt in ("f32", "bf16"):
        assert wgrad_name("bf16", False, E, S, S, N, K, dy_aligned=False, x_aligned=False,
                          out_dtype=odt) == ("wide256", 1)
        o = inside(np.zeros((E, N, K)), odt, shift)
        got = bsmm.bsmm_expert_wgrad(inside(dy, "bf16", shift), xg, og, fg, out_dtype=odt, out=o)
        assert np.array_equal(host(got), as_type(want, odt)), odt
        assert only_inside(o, shift)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("loads,N,K,name,parts", [
    (MANY, 1024, 1024, "wide192", 1), (MANY, 2048, 1024, "wide256", 1),
    (RAGGED, 1024, 1000, "wide128", 1), ([150, 0, 145], 136, 4096, "wide128", 16),
    ([150, 0, 145], 136, 4104, "wide128", 13)])
def test_wide_tiles_of_aligned_rows(loads, N, K, name, parts, back):
    rng = np.random.default_rng(N + K)
    off, S, E = sorted_offsets(loads), sum(loads) + 5, len(loads)
    order = rng.permutation(S).astype(np.int32)
    assert mm_name("bf16", back, E, S, N, K) == (name, parts)
    x, w = ints(rng, S, K, top=2), ints(rng, E, N, K, top=2)
    wg = dev(w.transpose(0, 2, 1).copy(), TDT["bf16"]).transpose(1, 2) if back else \
        dev(w, TDT["bf16"])
    for odt in ("f32", "bf16"):
        got = bsmm.bsmm_expert_mm(dev(x, TDT["bf16"]), wg, dev(order), dev(off), out_dtype=odt)
        assert np.array_equal(host(got), as_type(product(x, w, order, off), odt))


CKPT = [(16, 2048, 4, 1024, 1024, 1), (2, 3692, 2, 381, 2592, 5), (1, 9000, 2, 1024, 768, 16),
        (2, 6000, 4, 768, 1024, 10)]


@pytest.mark.parametrize("odt", ["bf16", "f32"])
@pytest.mark.parametrize("E,T,k,N,K,parts", CKPT)
def test_restored_checkpoints(E, T, k, N, K, parts, odt):
    """Codes and bytes in padded rows, a workspace of NaN, parts of the slots."""
    rng = np.random.default_rng(E + T)
    S = T * k
    expert = rng.integers(0, E + 1, S)                   # E: none
    order = np.argsort(expert, kind="stable").astype(np.int32)
    off = np.searchsorted(expert[order], np.arange(E + 1)).astype(np.int32)
    need = bsmm.bsmm_expert_wgrad_workspace_bytes("bf16", True, E, T, S, N, K)
    named = lambda room: wgrad_name("bf16", True, E, T, S, N, K, out_dtype=odt,  # noqa: E731
                                    dy_aligned=N % 4 == 0, workspace=room)
    assert named(None) == ("restored", parts) and named(T * K * 2 - 1)[0].startswith("tile")
    dy = ints(rng, S, N, top=1)
    q = rng.integers(-3, 4, (T, K)).astype(np.int8)
    byte = rng.integers(132, 134, (T, K // 32)).astype(np.uint8)
    x = X.restore(q, byte)
    want = np.zeros((E, N, K))
    for e in range(E):
        s = order[off[e]:off[e + 1]]
        want[e] = dy[s].astype(np.float64).T @ x[s // k]
    qg = torch.full((T, K + 40), 77, dtype=torch.int8, device=DEV)[:, 8:8 + K]
    qg.copy_(dev(q))
    sg = torch.full((T, K // 32 + 3), 255, dtype=torch.uint8, device=DEV)[:, 1:1 + K // 32]
    sg.copy_(dev(byte))
    nan = torch.full((need // 4 + 4,), float("nan"), device=DEV)
    for ws in (None, False, nan, nan[:T * K // 2]):
        got = bsmm.bsmm_expert_wgrad(dev(dy, TDT["bf16"]), qg, dev(order), dev(off), x_scale=sg,
                                     x_slots_per_row=k, out_dtype=odt, workspace=ws)
        assert np.array_equal(host(got), as_type(want, odt)), ws is None


@pytest.mark.parametrize("workspace", [None, False])
def test_restored_special_blocks(workspace):
    """A block of byte 255 makes its columns of its expert's gradient NaN and
    no others; one of byte 0 stands for codes of 2^-133, which a matrix
    instruction may flush."""
    E, T, k, N, K = 16, 2048, 4, 1024, 1024
    rng = np.random.default_rng(11)
    S = T * k
    order = rng.permutation(S).astype(np.int32)
    off = sorted_offsets([S // E] * E)
    name = wgrad_name("bf16", True, E, T, S, N, K, workspace=None if workspace is None else 0)[0]
    assert name == ("restored" if workspace is None else "tile128")
    dy = ints(rng, S, N, top=1)
    q = rng.integers(-3, 4, (T, K)).astype(np.int8)
    byte = np.full((T, K // 32), 133, np.uint8)
    byte[:, 7] = 0                                       # columns 224 .. 255
    byte[9, 3], q[9, 96:128] = 255, 0                    # four slots of token 9
    got = host(bsmm.bsmm_expert_wgrad(dev(dy, TDT["bf16"]), dev(q), dev(order), dev(off),
                                      x_scale=dev(byte), x_slots_per_row=k, workspace=workspace))
    hit = {int(np.searchsorted(off, i, "right")) - 1 for i in np.flatnonzero(order // k == 9)}
    clean = byte.copy()
    clean[9, 3] = 133
    x = X.restore(q, clean)
    for e in range(E):
        s = order[off[e]:off[e + 1]]
        d = dy[s].astype(np.float64)
        want = d.T @ x[s // k]
        if e in hit:
            assert np.isnan(got[e][:, 96:128]).all()
            got[e][:, 96:128] = want[:, 96:128]
        assert (np.abs(got[e][:, 224:256]) <= np.abs(d).sum(0)[:, None] * 3 * 2.0**-133).all()
        got[e][:, 224:256] = want[:, 224:256]
        assert np.array_equal(got[e], want)


FAR = [  # type, row stride from a multiple of 16 bytes, slots a row, kernel
    ("bf16", 0, 8, "wide256"), ("bf16", 1, 8, "tile64"), ("bf16", 1, 500, "wide128"),
    ("f32", 0, 12, "tile64"), ("f32", 1, 12, "tile64")]


@pytest.mark.parametrize("dt,odd,per,name", FAR)
def test_far_rows_of_the_tiles(dt, odd, per, name):
    """Rows of x and of out, of the weight and across it, past 2^31 elements."""
    rng = np.random.default_rng(per)
    t, R = TDT[dt], 3
    N, K = (64, 72) if per < 500 else (2048, 1100)
    S = R * per
    off = sorted_offsets([S])
    xh, wh = ints(rng, R, K, top=2), ints(rng, 1, N, K, top=2)
    assert mm_name(dt, False, 1, S, N, K, aligned=not odd, workspace=0) == (name, 1)
    want = product(xh, wh, None, off, per)
    x = far((R, K), 2**30 + 64 + odd, t)
    x.copy_(dev(xh))
    out = far((S, N), (2**31 // S + 64) // 8 * 8 + 64 + odd, torch.float32)
    w = dev(wh, t)
    got = bsmm.bsmm_expert_mm(x, w, None, dev(off), slots_per_row=per, out=out, out_dtype="f32",
                              workspace=False)
    assert np.array_equal(host(got), want)
    del out, got
    x = inside(xh, dt, odd, 8 - odd)
    for across in (False, True):
        rows, cols = (K, N) if across else (N, K)
        wg = far((rows, cols), (2**31 // rows + 64) // 8 * 8 + 64 + odd, t)
        wg.copy_(dev(wh[0].T.copy() if across else wh[0]))
        wg = (wg.t() if across else wg).unsqueeze(0)
        got = bsmm.bsmm_expert_mm(x, wg, None, dev(off), slots_per_row=per, out_dtype="f32",
                                  workspace=False)
        assert np.array_equal(host(got), want), across
        del wg


@pytest.mark.parametrize("dt,codes,odd,name", [("bf16", False, 0, "wide256"),
                                               ("bf16", False, 1, "wide256"),
                                               ("bf16", True, 0, "restored"),
                                               ("bf16", True, 1, "tile128"),
                                               ("f32", False, 0, "tile128"),
                                               ("f32", True, 0, "tile128")])
def test_far_rows_of_the_gradients_tiles(dt, codes, odd, name):
    rng = np.random.default_rng(odd + 2 * codes)
    t, R, per, N, K = TDT[dt], 3, 1500, 2048, 2048
    S = R * per
    off = sorted_offsets([S])
    workspace = None if name == "restored" else False
    assert wgrad_name(dt, codes, 1, R, S, N, K, dy_aligned=not odd, x_aligned=not odd,
                      workspace=None if workspace is None else 0)[0] == name
    dyh, xh = ints(rng, R, N, top=1), ints(rng, R, K, top=1)
    dy, x = far((R, N), 2**30 + 64 + odd, t), far((R, K), 2**30 + 64 + odd,
                                                  torch.int8 if codes else t)
    dy.copy_(dev(dyh))
    x.copy_(dev(xh))
    scale = torch.full((R, K // 32), 133, dtype=torch.uint8, device=DEV) if codes else None
    dw = far((N, K), 2**20 + 64 + odd, torch.float32).unsqueeze(0)
    got = bsmm.bsmm_expert_wgrad(dy, x, None, dev(off), x_scale=scale, dy_slots_per_row=per,
                                 x_slots_per_row=per, out=dw, workspace=workspace)
    assert np.array_equal(host(got)[0], per * (dyh.astype(np.float64).T @ xh))


def test_the_same_bits_whatever_the_workspace_holds():
    """With the bytes of the query, with many more, after a larger call and in
    a graph: the same order of sums."""
    S, N, K = 804, 2872, 3136
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(S, K, generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randn(1, K, N, generator=g, device=DEV).to(torch.bfloat16).transpose(1, 2)
    off = dev(np.array([0, S], np.int32))
    need = bsmm.bsmm_expert_mm_workspace_bytes("bf16", True, 1, S, N, K)
    assert need > 0

    def call(ws=None):
        return bsmm.bsmm_expert_mm(x, w, None, off, out_dtype="f32", workspace=ws)

    first = call()
    for size in (need, 2 * need, 2**28):
        assert torch.equal(call(torch.empty(size, dtype=torch.uint8, device=DEV)), first), size
    big = torch.zeros(64, 60000, dtype=torch.bfloat16, device=DEV)
    bsmm.bsmm_expert_mm(big, torch.zeros(1, 8000, 60000, dtype=torch.bfloat16, device=DEV), None,
                        dev(np.array([0, 64], np.int32)))
    assert torch.equal(call(), first)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = call()
    for _ in range(3):
        static.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(static, first)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("back", [False, True])
def test_no_columns_give_zeros_whatever_the_scale(back, dt):
    scale = torch.tensor([1.0, float("inf"), float("nan"), -1.0, float("-inf"), 0.0], device=DEV)
    x = torch.empty(6, 0, device=DEV, dtype=TDT[dt])
    w = torch.empty(2, 0, 40, device=DEV, dtype=TDT[dt]).transpose(1, 2) if back else \
        torch.empty(2, 40, 0, device=DEV, dtype=TDT[dt])
    for odt in ("f32", "bf16"):
        out = torch.full((6, 40), float("nan"), device=DEV, dtype=TDT[odt])
        bsmm.bsmm_expert_mm(x, w, None, dev(np.array([0, 3, 5], np.int32)), row_scale=scale,
                            out_dtype=odt, out=out)
        assert not host(out).any()
