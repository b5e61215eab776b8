"""4-bit weights on the GPU: the quantiser's codes, scales, zero points and
values bit for bit against the oracle, and the products dense and routed.

Products are checked twice.  On small integers with power-of-two scales every
partial sum is a multiple of 2**-4 below 2**19, so any order of fp32 additions
is exact and the results must be equal: that pins indexing, groups, zero
points, odd edges and routing.  On normal data the error is bounded from the
sums: over a group of G the partial sums of (16 + code) x and of x times (16 +
zero) have a size of about 22 sqrt(G) each, an fp32 addition errs by at most
2**-23 of that (truncation), and G of them add up as independent errors to
2**-23 * 22 * G * sqrt(2) / sqrt(3); against the group's share of the result,
4.6 sqrt(G), that is 2**-23 * 3.9 * sqrt(G), 5.3e-6 at G = 128, in the
Frobenius norm, and 1e-4 of the result's rms leaves an element 19 times that.
A bf16 output must be the fp32 output of the same call rounded to nearest even.
(The kernels sum (code - zero) x, which errs less than these two sums: this
limit is an upper one, test_gpu_w4_accuracy.py has theirs.)
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


def dev(a, dt=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dt is None else t.to(dt)


def host(t):
    torch.cuda.synchronize()
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


# --------------------------------------------------------------- quantiser --

def weights(R, K, seed):
    rng = np.random.default_rng(seed)
    w = rng.standard_normal((R, K)) * np.exp2(rng.integers(-30, 30, (R, 1)))
    w[rng.random((R, K)) < 0.05] = 0.0
    w[:, ::17] *= 8
    # groups of one sign, of zeros, of values whose scale underflows, of ties
    w[0] = np.abs(w[0])
    if R > 4:
        w[1] = -np.abs(w[1])
        w[2] = 0.0
        w[3] = 1e-44
        w[4] = np.arange(K) % 15 - 7 + 0.5
        w[4, ::16] = 7
    return w.astype(np.float32)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("sym", [True, False])
@pytest.mark.parametrize("dt,st", [("bf16", "f32"), ("f32", "bf16"), ("f32", "f32"),
                                   ("bf16", "bf16")])
def test_quantiser_exact(group, sym, dt, st):
    for R, K in ((1, group), (7, 3 * group), (37, 1024), (5, 4096 + group)):
        w = dev(weights(R, K, R * K), TDT[dt])
        q, s, z, v = bsmm.bsmm_quant_w4(w, group=group, symmetric=sym, scale_dtype=st,
                                        values=True)
        code, es, ez, ev = w4.quantise(host(w), group, sym, st)
        assert s.dtype == TDT[st] and np.array_equal(host(s), es)
        if sym:
            assert z is None
        else:
            assert np.array_equal(host(z), ez)
        assert np.array_equal(host(q), w4.pack(code)), (R, K)
        assert v.dtype == w.dtype
        assert np.array_equal(host(v), w4.bf16(ev) if dt == "bf16" else ev)


def test_quantiser_rows_and_batches():
    w = dev(weights(24, 512, 9))
    wide = torch.zeros(24, 520, device=DEV)
    wide[:, :512] = w
    a = bsmm.bsmm_quant_w4(w, group=64, symmetric=False)
    b = bsmm.bsmm_quant_w4(wide[:, :512], group=64, symmetric=False)
    c = bsmm.bsmm_quant_w4(w.view(4, 6, 512), group=64, symmetric=False)
    for x, y, t in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x, t.reshape(x.shape)) and t.shape[:2] == (4, 6)
    q, s, z = bsmm.bsmm_quant_w4(torch.empty(0, 64, device=DEV), group=64)
    assert q.shape == (0, 32) and s.shape == (0, 1) and z is None


# ---------------------------------------------------------------- products --

def integer_case(M, N, K, group, zero, dt, seed, E=None):
    """Integers in x, power-of-two scales: every sum is exact in fp32."""
    rng = np.random.default_rng(seed)
    lead = (N,) if E is None else (E, N)
    code = rng.integers(0, 16, lead + (K,))
    q = np.concatenate([w4.pack(c) for c in code.reshape(-1, N, K)]).reshape(lead + (K // 2,))
    s = np.exp2(rng.integers(-3, 1, lead + (K // group,))).astype(np.float32)
    z = rng.integers(0, 16, lead + (K // group,)).astype(np.uint8) if zero else None
    x = rng.integers(-3, 4, (M, K)).astype(np.float32)
    return dict(x=x, q=q, s=s, z=z)


def same(got, want, out):
    want = w4.bf16(want) if out == "bf16" else want
    g = host(got)
    assert g.shape == want.shape
    bad = np.argwhere(g != want)
    assert bad.size == 0, f"{len(bad)} differ, first {bad[:3].tolist()}"


def close(run, want):
    """run(out_dtype): the fp32 result against the oracle, the bf16 result
    against the fp32 one."""
    f = run("f32")
    g = host(f)
    assert g.shape == want.shape
    n, rms = np.linalg.norm(want), np.sqrt((want ** 2).mean())
    err = np.abs(g - want)
    assert np.linalg.norm(err) <= n * 2e-5
    assert (err <= 1e-4 * rms).all()
    assert torch.equal(run("bf16"), f.to(torch.bfloat16))


SHAPES = [(1, 1, 128), (1, 16, 256), (1, 257, 4096), (2, 100, 384), (5, 33, 8192), (16, 64, 1024),
          (17, 48, 640), (31, 130, 2048), (33, 17, 1152), (64, 257, 512), (65, 129, 1024),
          (127, 256, 768), (129, 320, 2048), (300, 200, 896), (513, 384, 640)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_mm_integers_exact(M, N, K, group):
    for i, (dt, st, zero, out) in enumerate((("bf16", "f32", True, "f32"),
                                             ("f32", "bf16", False, "f32"),
                                             ("bf16", "bf16", False, "bf16"),
                                             ("f32", "f32", True, "bf16"))):
        c = integer_case(M, N, K, group, zero, dt, M + N + K + i)
        y = bsmm.bsmm_w4_mm(dev(c["x"], TDT[dt]), dev(c["q"]), dev(c["s"], TDT[st]),
                            dev(c["z"]) if zero else None, out_dtype=out)
        same(y, w4.w4_mm(c["x"], c["q"], c["s"], c["z"]), out)


@pytest.mark.parametrize("group,K", [(32, 32), (32, 96), (32, 160), (32, 4128), (64, 64),
                                     (64, 192), (64, 2112), (128, 128)])
@pytest.mark.parametrize("M", [1, 40, 200])
def test_mm_short_and_ragged_k(group, K, M):
    for dt in ("bf16", "f32"):
        c = integer_case(M, 70, K, group, True, dt, K + M)
        y = bsmm.bsmm_w4_mm(dev(c["x"], TDT[dt]), dev(c["q"]), dev(c["s"]), dev(c["z"]),
                            out_dtype="f32")
        same(y, w4.w4_mm(c["x"], c["q"], c["s"], c["z"]), "f32")


@pytest.mark.parametrize("M", [1, 9, 50, 150])
def test_mm_strided(M):
    """Views with longer rows, a poisoned margin, one scale row for all."""
    c = integer_case(M, 96, 512, 128, True, "bf16", 77 + M)
    x = torch.full((M, 520), float("nan"), device=DEV, dtype=torch.bfloat16)
    x[:, :512] = dev(c["x"])
    q = torch.full((96, 272), 0xFF, device=DEV, dtype=torch.uint8)
    q[:, :256] = dev(c["q"])
    s = torch.full((96, 7), float("nan"), device=DEV)
    s[:, :4] = dev(c["s"])
    z = torch.full((96, 5), 255, device=DEV, dtype=torch.uint8)
    z[:, :4] = dev(c["z"])
    out = torch.full((M + 1, 101), -7.0, device=DEV)
    y = bsmm.bsmm_w4_mm(x[:, :512], q[:, :256], s[:, :4], z[:, :4], out_dtype="f32",
                        out=out[:M, :96])
    same(y, w4.w4_mm(c["x"], c["q"], c["s"], c["z"]), "f32")
    assert (out[:, 96:] == -7.0).all() and (out[M] == -7.0).all()
    one = dev(c["s"][:1]).expand(96, 4)
    y = bsmm.bsmm_w4_mm(x[:, :512], q[:, :256], one, None, out_dtype="f32")
    same(y, w4.w4_mm(c["x"], c["q"], np.repeat(c["s"][:1], 96, 0)), "f32")


@pytest.mark.parametrize("far", ["x", "w", "scale", "zero"])
@pytest.mark.parametrize("M,K,group", [(3, 288, 32), (5, 192, 64), (20, 256, 128)])
def test_mm_rows_far_apart(far, M, K, group):
    """Row strides whose multiples pass 31 bits."""
    N = 3
    c = integer_case(M, N, K, group, True, "bf16", K)
    ops = dict(x=dev(c["x"], torch.bfloat16), w=dev(c["q"]), scale=dev(c["s"]), zero=dev(c["z"]))
    t = ops[far]
    ld = (1 << (28 if far == "zero" else 27)) // t.element_size()
    rows = min(t.shape[0], 3)
    wide = torch.zeros(rows * ld, dtype=t.dtype, device=DEV).view(rows, ld)
    wide[:, :t.shape[1]] = t[:rows]
    ops[far] = wide[:, :t.shape[1]]
    if far == "x":
        c["x"] = c["x"][:rows]
    y = bsmm.bsmm_w4_mm(ops["x"], ops["w"], ops["scale"], ops["zero"], out_dtype="f32")
    same(y, w4.w4_mm(c["x"], c["q"], c["s"], c["z"]), "f32")


# sizes at which the cost rule takes tiles of 128 rows and of 256 (the last of
# each group of sizes), with one K step to several, odd edges, and for groups
# of 32 a last step of one group
TILES = [(32, 1100, 900, 32, "bf16"), (32, 1700, 1290, 352, "bf16"), (32, 1700, 1700, 352, "f32"),
         (32, 2047, 2100, 288, "bf16"), (64, 65, 100, 64, "bf16"), (64, 1290, 1100, 320, "bf16"),
         (64, 1030, 2300, 192, "f32"), (64, 2047, 2100, 448, "bf16"), (64, 2300, 2100, 128, "f32"),
         (128, 500, 1300, 128, "bf16"), (128, 1200, 1030, 256, "bf16"),
         (128, 1300, 1300, 384, "f32"), (128, 2047, 2100, 640, "bf16"),
         (128, 2049, 2100, 256, "f32")]


@pytest.mark.parametrize("group,M,N,K,dt", TILES)
def test_mm_tiles_integers_exact(group, M, N, K, dt):
    for st, zero, out in (("f32", True, "f32"), ("bf16", False, "bf16")):
        c = integer_case(M, N, K, group, zero, dt, M + K)
        y = bsmm.bsmm_w4_mm(dev(c["x"], TDT[dt]), dev(c["q"]), dev(c["s"], TDT[st]),
                            dev(c["z"]) if zero else None, out_dtype=out)
        same(y, w4.w4_mm(c["x"], c["q"], c["s"], c["z"]), out)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_mm_tiles_normal_data(group, dt):
    rng = np.random.default_rng(group)
    w = dev((rng.standard_normal((2051, 1024)) * 0.02).astype(np.float32))
    x = dev(rng.standard_normal((2047, 1024)).astype(np.float32), TDT[dt])
    for M, sym, st in ((800, True, "bf16"), (2047, False, "f32")):
        q, s, z = bsmm.bsmm_quant_w4(w, group=group, symmetric=sym, scale_dtype=st)
        close(lambda out: bsmm.bsmm_w4_mm(x[:M], q, s, z, out_dtype=out),
              w4.w4_mm(host(x[:M]), host(q), host(s), None if sym else host(z)))


def test_mm_degenerate():
    c = integer_case(3, 8, 64, 64, False, "bf16", 5)
    x, q, s = dev(c["x"], torch.bfloat16), dev(c["q"]), dev(c["s"])
    assert bsmm.bsmm_w4_mm(x[:0], q, s).shape == (0, 8)
    assert bsmm.bsmm_w4_mm(x, q[:0], s[:0]).shape == (3, 0)
    y = bsmm.bsmm_w4_mm(x[:, :0], q[:, :0], s[:, :0])
    assert y.shape == (3, 8) and (y == 0).all()


@pytest.mark.parametrize("M", [1, 13, 48, 90, 300])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_mm_normal_data(M, group, dt):
    rng = np.random.default_rng(M + group)
    x = dev(rng.standard_normal((M, 2048)).astype(np.float32), TDT[dt])
    w = dev((rng.standard_normal((515, 2048)) * 0.02).astype(np.float32))
    for sym, st in ((True, "bf16"), (False, "f32")):
        q, s, z = bsmm.bsmm_quant_w4(w, group=group, symmetric=sym, scale_dtype=st)
        close(lambda out: bsmm.bsmm_w4_mm(x, q, s, z, out_dtype=out),
              w4.w4_mm(host(x), host(q), host(s), None if sym else host(z)))


def test_mm_full_precision_activations():
    """fp32 activations keep all 24 bits: integers up to 2**14 + 1 in a
    32-element row give sums below 2**24."""
    rng = np.random.default_rng(8)
    for M in (1, 20, 140):
        c = integer_case(M, 40, 32, 32, True, "f32", M)
        c["x"] = rng.integers(-2**14, 2**14 + 1, (M, 32)).astype(np.float32)
        c["s"][:] = 1.0
        c["x"][:, 4:] = 0
        y = bsmm.bsmm_w4_mm(dev(c["x"]), dev(c["q"]), dev(c["s"]), dev(c["z"]), out_dtype="f32")
        same(y, w4.w4_mm(c["x"], c["q"], c["s"], c["z"]), "f32")
        # single elements with odd low bits: one product per output
        x = np.zeros((M, 32), np.float32)
        x[np.arange(M), np.arange(M) % 32] = (2**20 + 2 * np.arange(M) + 1) * 2.0**-9
        y = bsmm.bsmm_w4_mm(dev(x), dev(c["q"]), dev(c["s"]), None, out_dtype="f32")
        err = np.abs(host(y) - w4.w4_mm(x, c["q"], c["s"]))
        # three truncating additions of 31 x, one rounding of 24 x, x < 2**11 + 1
        assert (err <= 2.0**11 * 256 * 2.0**-24).all()


# ------------------------------------------------------------------ routed --

def routing(T, k, E, seed, unused=0.0):
    """Slots sorted by expert, stable; a share of them without an expert."""
    rng = np.random.default_rng(seed)
    e = np.stack([rng.permutation(E)[:k] for _ in range(T)]) if T else np.zeros((0, k), int)
    e = np.minimum(e, rng.integers(0, E, 1) + E // 2)          # uneven loads, empty experts
    e = np.where(rng.random(e.shape) < unused, E, e).reshape(-1)
    order = np.argsort(e, kind="stable").astype(np.int32)
    offsets = np.searchsorted(np.sort(e), np.arange(E + 1)).astype(np.int32)
    return order, offsets


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (3, 2, 5), (16, 4, 8), (33, 4, 16),
                                   (70, 6, 130), (200, 2, 4), (300, 8, 9), (5, 2, 1000)])
@pytest.mark.parametrize("second", [False, True])
def test_expert_integers_exact(T, k, E, second):
    N, K = (40, 192) if E < 100 else (24, 64)
    for i, (dt, group, zero, out, unused) in enumerate((("bf16", 32, True, "f32", 0.0),
                                                        ("f32", 64, False, "f32", 0.3),
                                                        ("bf16", 64, True, "bf16", 1.0))):
        order, offsets = routing(T, k, E, T + E + i, unused)
        c = integer_case(T * k if second else T, N, K, group, zero, dt, T + i, E)
        rs = np.exp2(np.random.default_rng(i).integers(-2, 2, T * k)).astype(np.float32)
        out_t = torch.full((T * k, N), 9.0, device=DEV, dtype=TDT[out])
        y = bsmm.bsmm_w4_expert_mm(
            dev(c["x"], TDT[dt]), dev(c["q"]), dev(c["s"]), dev(c["z"]) if zero else None,
            dev(order), dev(offsets), slots_per_row=1 if second else k,
            row_scale=dev(rs) if second else None, out_dtype=out, out=out_t)
        same(y, w4.w4_expert_mm(c["x"], c["q"], c["s"], c["z"], order, offsets,
                                1 if second else k, rs if second else None), out)


@pytest.mark.parametrize("group,K,dt", [(32, 352, "bf16"), (64, 320, "bf16"), (64, 320, "f32"),
                                        (128, 128, "bf16"), (128, 640, "bf16")])
def test_expert_tiles_integers_exact(group, K, dt):
    """Sizes at which the cost rule takes tiles of 128 rows."""
    T, k, E, N = 500, 4, 8, 1500
    for i, (second, unused) in enumerate(((False, 0.0), (True, 0.3))):
        order, offsets = routing(T, k, E, 5 + i, unused)
        c = integer_case(T * k if second else T, N, K, group, second, dt, K + i, E)
        rs = np.exp2(np.random.default_rng(i).integers(-2, 2, T * k)).astype(np.float32)
        y = bsmm.bsmm_w4_expert_mm(
            dev(c["x"], TDT[dt]), dev(c["q"]), dev(c["s"]), dev(c["z"]) if second else None,
            dev(order), dev(offsets), slots_per_row=1 if second else k,
            row_scale=dev(rs) if second else None, out_dtype="f32")
        same(y, w4.w4_expert_mm(c["x"], c["q"], c["s"], c["z"], order, offsets,
                                1 if second else k, rs if second else None), "f32")


@pytest.mark.parametrize("group", [32, 128])
def test_expert_normal_data(group):
    T, k, E, N, K = 500, 4, 6, 200, 1024
    rng = np.random.default_rng(group)
    order, offsets = routing(T, k, E, 3)
    w = dev((rng.standard_normal((E, N, K)) * 0.02).astype(np.float32))
    q, s, z = bsmm.bsmm_quant_w4(w, group=group, symmetric=False)
    for dt in ("bf16", "f32"):
        x = dev(rng.standard_normal((T, K)).astype(np.float32), TDT[dt])
        close(lambda out: bsmm.bsmm_w4_expert_mm(x, q, s, z, dev(order), dev(offsets),
                                                 slots_per_row=k, out_dtype=out),
              w4.w4_expert_mm(host(x), host(q), host(s), host(z), order, offsets, k))


def test_expert_no_slots():
    c = integer_case(2, 8, 64, 64, False, "bf16", 5, 3)
    y = bsmm.bsmm_w4_expert_mm(dev(c["x"], torch.bfloat16), dev(c["q"]), dev(c["s"]), None,
                               torch.empty(0, dtype=torch.int32, device=DEV),
                               torch.zeros(4, dtype=torch.int32, device=DEV))
    assert y.shape == (0, 8)


def test_expert_lists_out_of_range():
    """Slots, rows and offsets past the arrays touch nothing outside them;
    the rows of the sound slots are right."""
    E, N, K, S = 3, 32, 64, 12
    c = integer_case(S, N, K, 64, False, "bf16", 6, E)
    order = np.arange(S, dtype=np.int32)
    order[[2, 7]] = [-5, 1 << 30]
    offsets = np.array([0, 4, 8, 1 << 29], np.int32)
    guard = torch.full((S + 8, N), -3.0, device=DEV)
    bsmm.bsmm_w4_expert_mm(dev(c["x"], torch.bfloat16), dev(c["q"]), dev(c["s"]), None, dev(order),
                           dev(offsets), out_dtype="f32", out=guard[4:4 + S])
    want = w4.w4_expert_mm(c["x"], c["q"], c["s"], None, np.arange(S), [0, 4, 8, 12])
    got = host(guard)
    keep = [i for i in range(S) if i not in (2, 7)]
    assert np.array_equal(got[4:4 + S][keep], want[keep])
    assert (got[:4] == -3).all() and (got[4 + S:] == -3).all()
    assert (got[[6, 11]] == -3).all()


def test_expert_many_slots():
    """More items than one launch holds, and offsets that fall: 512 runs of
    all 2^27 slots count 2^32 blocks of 16 rows, and nothing outside the
    arrays may be touched."""
    E, K, S = 1024, 32, 1 << 27
    c = integer_case(1, 1, K, 32, False, "f32", 15, E)
    x, q, s = dev(c["x"]), dev(c["q"]), dev(c["s"])
    order = torch.arange(S, dtype=torch.int32, device=DEV).flip(0).contiguous()
    guard = torch.full((S + 2048, 1), -3.0, device=DEV)
    out = guard[1024:1024 + S]
    ends = np.sort(np.random.default_rng(1).integers(0, S + 1, E + 1)).astype(np.int32)
    ends[0] = 0
    each = dev(w4.w4_expert_mm(c["x"], c["q"], c["s"], None, np.arange(E), np.arange(E + 1), E)
               .astype(np.float32))
    bsmm.bsmm_w4_expert_mm(x, q, s, None, order, dev(ends), slots_per_row=S, out_dtype="f32",
                           out=out)
    want = torch.cat([torch.repeat_interleave(each, dev(np.diff(ends).astype(np.int64)), 0),
                      torch.zeros(S - int(ends[-1]), 1, device=DEV)])
    assert torch.equal(out, want.flip(0))
    ends[::2], ends[1::2] = 0, S
    bsmm.bsmm_w4_expert_mm(x, q, s, None, order, dev(ends), slots_per_row=S, out_dtype="f32",
                           out=out)
    assert (guard[:1024] == -3).all() and (guard[1024 + S:] == -3).all()


# ----------------------------------------------------- streams and graphs --

@pytest.mark.parametrize("M", [1, 40, 200])
def test_stream_and_graph(M):
    c = integer_case(M, 64, 512, 128, True, "bf16", 21)
    x, q, s, z = dev(c["x"], torch.bfloat16), dev(c["q"]), dev(c["s"]), dev(c["z"])
    want = w4.w4_mm(c["x"], c["q"], c["s"], c["z"])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    y = bsmm.bsmm_w4_mm(x, q, s, z, out_dtype="f32", stream=st)
    st.synchronize()
    same(y, want, "f32")
    out = torch.zeros(M, 64, device=DEV)
    g = torch.cuda.CUDAGraph()
    bsmm.bsmm_w4_mm(x, q, s, z, out_dtype="f32", out=out)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        bsmm.bsmm_w4_mm(x, q, s, z, out_dtype="f32", out=out)
    for i in range(3):
        x.copy_(dev(c["x"], torch.bfloat16) * (i + 1))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        same(out, want * (i + 1), "f32")
