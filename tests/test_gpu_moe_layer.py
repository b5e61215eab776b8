"""The operators together, as the example layer runs them: outputs and the
router's gradient against the plain layer in 64 bits on the CPU, which makes
the same choices.

Tolerances: the layer rounds h and its gated product to bf16 (2**-9 relative
each, independent between elements), which the plain layer does not; an output
is a sum of F such products, so its error is at most about sqrt(2) * 2 * 2**-9
of the output's rms in the Frobenius norm (a gated product has two rounded
factors): 5.5e-3, doubled for the few terms that dominate a row.  The gradient is
linear in the layer's output rows, with the same relative error.
"""

import os
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
TOL = 1.1e-2


@pytest.fixture(autouse=True)
def _lib(gpu_lib):
    yield


def plain(layer, x, router, index, mask, alpha):
    """(out, loss) in 64 bits; the choice is given, router has a gradient."""
    d = {n: getattr(layer, n + "_values").double().cpu() for n in ("w_in", "w_out", "s_in",
                                                                   "s_out")}

    def gate(h):
        a, b = h.chunk(2, -1)
        return torch.nn.functional.silu(a) * b

    T, E, k = x.shape[0], layer.E, layer.k
    p = torch.softmax(x @ router.t(), 1)
    keep = torch.ones(T, dtype=torch.bool) if mask is None else mask
    w = torch.gather(p, 1, index.clamp(min=0))
    w = w / w.sum(1, keepdim=True) * keep[:, None]
    out = []
    for t in range(T):
        y = gate(x[t] @ d["s_in"].t()) @ d["s_out"].t()
        for j in range(k):
            if keep[t]:
                e = int(index[t, j])
                y = y + w[t, j] * (gate(x[t] @ d["w_in"][e].t()) @ d["w_out"][e].t())
        out.append(y)
    counts = torch.bincount(index[keep].reshape(-1), minlength=E).double()
    L = int(keep.sum())
    loss = alpha * E / (k * L * L) * (counts * p[keep].sum(0)).sum()
    return torch.stack(out), loss


@pytest.mark.parametrize("T,D,F,E,k,group", [(1, 256, 128, 8, 2, 64), (37, 384, 256, 16, 4, 128),
                                             (130, 128, 64, 5, 5, 32)])
def test_layer_and_router_gradient(T, D, F, E, k, group):
    from moe_layer import MoeLayer
    layer = MoeLayer(D, F, E, k, group=group, seed=T)
    rng = np.random.default_rng(T)
    x = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    dout = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).cuda()
    mask = (torch.arange(T) < max(1, T - 3)).cuda()
    out, saved = layer(x, mask=mask, alpha=0.3)
    grad = layer.router_gradient(saved, dout)
    r = saved[2]
    served, _ = layer(x, mask=mask)
    torch.cuda.synchronize()

    router = layer.router.double().cpu().requires_grad_(True)
    want, loss = plain(layer, x.double().cpu(), router, r.index.long().cpu(), mask.cpu(), 0.3)
    ((want * dout.double().cpu()).sum() + loss).backward()
    assert (r.index[mask] >= 0).all() and (r.index[~mask] == -1).all()

    def off(got, ref):
        return float((got.double().cpu() - ref).norm() / ref.norm())

    assert off(out, want.detach()) < TOL
    assert off(served, want.detach()) < TOL
    assert off(grad, router.grad) < TOL
    assert abs(r.loss.item() - loss.item()) < 1e-5 * loss.item()
