"""The 4-bit operations and the router refuse tensors that are not all on one
GPU, before the library is called (no GPU needed: tensors that say they are
on one stand for those)."""

import pytest
import torch

import block_scaled_precision_gemm_amd as bsmm


class OnGpu(torch.Tensor):
    def get_device(self):
        return self.index

    index = 0


class OnAnotherGpu(OnGpu):
    index = 1


U8, I = torch.uint8, torch.int32
CALLS = {
    "quant": (lambda **a: bsmm.bsmm_quant_w4(a["w"]), dict(w=torch.zeros(4, 128))),
    "mm": (lambda **a: bsmm.bsmm_w4_mm(**a), dict(
        x=torch.zeros(2, 128), w=torch.zeros(8, 64, dtype=U8), scale=torch.zeros(8, 1),
        zero=torch.zeros(8, 1, dtype=U8), out=torch.zeros(2, 8, dtype=torch.bfloat16),
        workspace=torch.zeros(64))),
    "experts": (lambda **a: bsmm.bsmm_w4_expert_mm(**a), dict(
        x=torch.zeros(2, 128), w=torch.zeros(3, 8, 64, dtype=U8), scale=torch.zeros(3, 8, 1),
        zero=torch.zeros(3, 8, 1, dtype=U8), order=torch.zeros(2, dtype=I),
        offsets=torch.zeros(4, dtype=I), row_scale=torch.zeros(2),
        out=torch.zeros(2, 8, dtype=torch.bfloat16), workspace=torch.zeros(64))),
    "route": (lambda **a: bsmm.bsmm_route_topk(k=2, **a), dict(
        logits=torch.zeros(100, 8), mask=torch.ones(100, dtype=U8), workspace=torch.zeros(4096))),
    "back": (lambda **a: bsmm.bsmm_route_topk_backward(**a), dict(
        logits=torch.zeros(4, 8), index=torch.zeros(4, 2, dtype=I), weight=torch.zeros(4, 2),
        counts=torch.zeros(8, dtype=I), live=torch.zeros(1, dtype=I), dweight=torch.zeros(4, 2),
        dloss=torch.zeros(1), mask=torch.ones(4, dtype=torch.bool), out=torch.zeros(4, 8))),
}


@pytest.fixture(autouse=True)
def library(monkeypatch):
    """No call may get as far as the library."""
    class Called(Exception):
        pass

    class Library:
        def __getattr__(self, name):
            raise Called(name)

    monkeypatch.setattr(bsmm, "load", Library)
    monkeypatch.setattr(bsmm, "_stream", lambda stream: 0)
    return Called


@pytest.mark.parametrize("name", CALLS)
def test_all_on_the_host(name):
    call, args = CALLS[name]
    with pytest.raises(ValueError, match="must be on one GPU"):
        call(**args)


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("where", [torch.Tensor, OnAnotherGpu])
def test_one_elsewhere(name, where, library):
    call, args = CALLS[name]
    on = {n: t.as_subclass(OnGpu) for n, t in args.items()}
    with pytest.raises(library):        # nothing else is wrong with these
        call(**on)
    for n in args:
        if len(args) > 1:
            with pytest.raises(ValueError, match="must be on one GPU"):
                call(**{**on, n: args[n].as_subclass(where)})


def test_unused_arguments_of_the_gradient(library):
    """What no kernel will read may be anywhere."""
    call, args = CALLS["back"]
    on = {n: t.as_subclass(OnGpu) for n, t in args.items()}
    with pytest.raises(library):
        call(**{**on, "dweight": None, "weight": args["weight"]})
    with pytest.raises(library):
        call(**{**on, "dloss": None, "counts": args["counts"], "live": args["live"]})
