"""Single rows whose row stride is not a row's length: it is never used, and
a column of one element transposed is such a row."""

import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_amd as bsmm
from oracle import route as R, w4
from test_gpu_route import check_forward, logits
from test_gpu_w4 import dev, host, integer_case, same

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(gpu_lib):
    yield


def row(t):
    """The tensor [.., 1, n] with the strides of a transposed column."""
    c = t.contiguous().as_strided(t.shape, (*t.stride()[:-2], 1, 1))
    assert torch.equal(c, t)
    return c


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_products(group, dt):
    K = 256
    c = integer_case(1, 1, K, group, True, "f32", 1)
    ops = [row(dev(c["q"])), row(dev(c["s"])), row(dev(c["z"]))]
    x = row(dev(c["x"], dt))
    same(bsmm.bsmm_w4_mm(x, *ops, out_dtype="f32"), w4.w4_mm(c["x"], c["q"], c["s"], c["z"]),
         "f32")
    c = integer_case(1, 40, K, group, False, "f32", 2)
    out = row(torch.zeros(1, 40, device=x.device))
    bsmm.bsmm_w4_mm(row(dev(c["x"], dt)), dev(c["q"]), dev(c["s"]), out_dtype="f32", out=out)
    same(out, w4.w4_mm(c["x"], c["q"], c["s"]), "f32")
    # one expert with rows of its own, one row for all slots
    c = integer_case(1, 1, K, group, True, "f32", 3, 1)
    y = bsmm.bsmm_w4_expert_mm(row(dev(c["x"], dt)), row(dev(c["q"])), row(dev(c["s"])),
                               row(dev(c["z"])), dev(np.arange(3, dtype=np.int32)),
                               dev(np.array([0, 3], np.int32)), slots_per_row=3, out_dtype="f32")
    same(y, w4.w4_expert_mm(c["x"], c["q"], c["s"], c["z"], np.arange(3), [0, 3], 3), "f32")


def test_one_expert_of_a_strided_pair():
    """The stride of a single expert may be anything."""
    c = integer_case(2, 8, 64, 32, True, "f32", 4, 1)
    ops = [dev(c[n])[0][None].as_strided(c[n].shape, (7, c[n].shape[2], 1)) for n in "qsz"]
    y = bsmm.bsmm_w4_expert_mm(dev(c["x"]), *ops, dev(np.arange(2, dtype=np.int32)),
                               dev(np.array([0, 2], np.int32)), out_dtype="f32")
    same(y, w4.w4_expert_mm(c["x"], c["q"], c["s"], c["z"], np.arange(2), [0, 2]), "f32")


def test_quantiser():
    w = dev(np.random.default_rng(5).standard_normal((1, 256)).astype(np.float32))
    for a, b in zip(bsmm.bsmm_quant_w4(w, group=64, symmetric=False, values=True),
                    bsmm.bsmm_quant_w4(row(w), group=64, symmetric=False, values=True)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_router(dt):
    l = logits(1, 40, dt, 6)
    x = row(dev(l, torch.bfloat16 if dt == "bf16" else torch.float32))
    r = bsmm.bsmm_route_topk(x, 4, alpha=1.0)
    check_forward(r, R.route(l, 4, alpha=1.0))
    d = [bsmm.bsmm_route_topk_backward(t, r.index, r.weight, r.counts, r.live, dweight=r.weight,
                                       dloss=torch.ones(1, device=x.device), alpha=1.0, out=o)
         for t, o in ((x, row(torch.zeros_like(x))), (x.contiguous().clone(), None))]
    assert torch.equal(*d) and np.isfinite(host(d[0])).all()
