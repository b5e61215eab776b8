"""What the binding of the experts' products, the checkpoints and the gate
refuses before it calls the library (no GPU needed)."""

import pytest
import torch

import block_scaled_precision_gemm_amd as bsmm


class OnGpu(torch.Tensor):
    """Says that it is on GPU `index`; its views do too."""
    index = 0

    def get_device(self):
        return self.index


class OnAnotherGpu(OnGpu):
    index = 1


def t(*shape, dt=torch.bfloat16):
    return torch.zeros(*shape, dtype=dt).as_subclass(OnGpu)


U8, I8, F, I, H = torch.uint8, torch.int8, torch.float32, torch.int32, torch.float16

mm, wgrad = bsmm.bsmm_expert_mm, bsmm.bsmm_expert_wgrad
quant, gate, back = bsmm.bsmm_quant_int8_mx, bsmm.bsmm_swiglu, bsmm.bsmm_swiglu_backward


@pytest.mark.parametrize("call", [
    lambda: mm(t(4, 8, dt=H), t(2, 6, 8, dt=H), t(8, dt=I), t(3, dt=I)),
    lambda: mm(t(8), t(2, 6, 8), t(8, dt=I), t(3, dt=I)),
    lambda: mm(t(4, 8), t(6, 8), t(8, dt=I), t(3, dt=I)),
    lambda: mm(t(4, 8), t(2, 6, 8, dt=F), t(8, dt=I), t(3, dt=I)),
    lambda: mm(t(4, 8), t(2, 6, 9), t(8, dt=I), t(3, dt=I)),
    lambda: mm(t(8, 4).t(), t(2, 6, 8), t(8, dt=I), t(3, dt=I)),
    lambda: mm(t(4, 8), t(2, 6, 16)[:, :, ::2], t(8, dt=I), t(3, dt=I)),
    lambda: mm(t(4, 8), t(2, 6, 8), t(8, dt=F), t(3, dt=I)),
    lambda: mm(t(4, 8), t(2, 6, 8), t(2, 4, dt=I), t(3, dt=I)),
    lambda: mm(t(4, 8), t(2, 6, 8), t(8, dt=I), t(2, dt=I)),
    lambda: mm(t(4, 8), t(2, 6, 8), t(8, dt=I), t(3, dt=F)),
    lambda: mm(t(4, 8), t(2, 6, 8), t(16, dt=I)[::2], t(3, dt=I)),
    lambda: mm(t(4, 8), t(2, 6, 8), t(8, dt=I), t(3, dt=I), slots_per_row=0),
    lambda: mm(t(4, 8), t(2, 6, 8), t(8, dt=I), t(3, dt=I), slots_per_row=2**31),
    lambda: mm(t(4, 8), t(2, 6, 8), t(8, dt=I), t(3, dt=I), row_scale=t(8)),
    lambda: mm(t(4, 8), t(2, 6, 8), t(8, dt=I), t(3, dt=I), row_scale=t(4, dt=F)),
    lambda: mm(t(4, 8), t(2, 6, 8), t(8, dt=I), t(3, dt=I), out_dtype="i32"),
    lambda: mm(t(4, 8), t(2, 6, 8), t(8, dt=I), t(3, dt=I), out=t(4, 6)),
    lambda: mm(t(4, 8), t(2, 6, 8), t(8, dt=I), t(3, dt=I), out=t(8, 6, dt=F)),
    lambda: mm(t(4, 8), t(2, 6, 8), t(8, dt=I), t(3, dt=I), out=t(6, 8).t()),
    lambda: wgrad(t(8, 6, dt=H), t(8, 8, dt=H), t(8, dt=I), t(3, dt=I)),
    lambda: wgrad(t(8, 6), t(8, 8, dt=F), t(8, dt=I), t(3, dt=I)),
    lambda: wgrad(t(8, 6), t(8, 32, dt=I8), t(8, dt=I), t(3, dt=I)),
    lambda: wgrad(t(8, 6), t(8, 32), t(8, dt=I), t(3, dt=I), x_scale=t(8, 1, dt=U8)),
    lambda: wgrad(t(8, 6), t(8, 40, dt=I8), t(8, dt=I), t(3, dt=I), x_scale=t(8, 1, dt=U8)),
    lambda: wgrad(t(8, 6), t(8, 64, dt=I8), t(8, dt=I), t(3, dt=I), x_scale=t(8, 1, dt=U8)),
    lambda: wgrad(t(8, 6), t(8, 64, dt=I8), t(8, dt=I), t(3, dt=I), x_scale=t(8, 2, dt=F)),
    lambda: wgrad(t(8, 6), t(8, 64, dt=I8), t(8, dt=I), t(3, dt=I), x_scale=t(2, 8, dt=U8).t()),
    lambda: wgrad(t(6, 8).t(), t(8, 8), t(8, dt=I), t(3, dt=I)),
    lambda: wgrad(t(8, 6), t(8, 8).t(), t(8, dt=I), t(3, dt=I)),
    lambda: wgrad(t(8, 6), t(8, 8), t(8, dt=I), t(3, 1, dt=I)),
    lambda: wgrad(t(8, 6), t(8, 8), t(8, dt=I), t(0, dt=I)),
    lambda: wgrad(t(8, 6), t(8, 8), t(8, dt=I), t(3, dt=I), dy_slots_per_row=0),
    lambda: wgrad(t(8, 6), t(8, 8), t(8, dt=I), t(3, dt=I), x_slots_per_row=-1),
    lambda: wgrad(t(8, 6), t(8, 8), t(8, dt=I), t(3, dt=I), out=t(2, 6, 8)),
    lambda: wgrad(t(8, 6), t(8, 8), t(8, dt=I), t(3, dt=I), out=t(2, 8, 6, dt=F).transpose(1, 2)),
    lambda: quant(t(4, 64, dt=H)), lambda: quant(t(64)), lambda: quant(t(4, 40)),
    lambda: quant(t(64, 4).t()),
    lambda: gate(t(4, 64, dt=H)), lambda: gate(t(64)), lambda: gate(t(4, 32)),
    lambda: gate(t(64, 64).t()), lambda: gate(t(4, 64), out=t(4, 64)),
    lambda: back(t(4, 32, dt=H), t(4, 64, dt=I8), t(4, 2, dt=U8)),
    lambda: back(t(4, 40), t(4, 80, dt=I8), t(4, 2, dt=U8)),
    lambda: back(t(4, 32), t(4, 64, dt=U8), t(4, 2, dt=U8)),
    lambda: back(t(4, 32), t(4, 32, dt=I8), t(4, 2, dt=U8)),
    lambda: back(t(4, 32), t(4, 64, dt=I8), t(4, 1, dt=U8)),
    lambda: back(t(4, 32), t(4, 64, dt=I8), t(4, 2, dt=I8)),
    lambda: back(t(4, 32), t(4, 64, dt=I8), t(4, 2, dt=U8), row_scale=t(4)),
    lambda: back(t(4, 32), t(4, 64, dt=I8), t(4, 2, dt=U8), row_scale=t(3, dt=F)),
    lambda: back(t(32, 4).t(), t(4, 64, dt=I8), t(4, 2, dt=U8)),
])
def test_rejects(call):
    with pytest.raises(ValueError):
        call()


CALLS = {
    "mm": (lambda **a: mm(**a), dict(x=t(4, 8), w=t(2, 6, 8), order=t(8, dt=I), offsets=t(3, dt=I),
                                     row_scale=t(8, dt=F), out=t(8, 6),
                                     workspace=t(64, dt=U8))),
    "wgrad": (lambda **a: wgrad(**a), dict(dy=t(8, 6), x=t(8, 32, dt=I8), x_scale=t(8, 1, dt=U8),
                                           order=t(8, dt=I), offsets=t(3, dt=I),
                                           out=t(2, 6, 32, dt=F),
                                           workspace=t(64, dt=U8))),
    "quant": (lambda **a: quant(**a), dict(x=t(4, 32))),
    "gate": (lambda **a: gate(**a), dict(h=t(4, 64), out=t(4, 32))),
    "back": (lambda **a: back(**a), dict(da=t(4, 32), q=t(4, 64, dt=I8), scale=t(4, 2, dt=U8),
                                         row_scale=t(4, dt=F))),
}


@pytest.mark.parametrize("name,arg", [(n, a) for n, (_, args) in CALLS.items() for a in args])
def test_every_tensor_is_on_the_gpu(name, arg):
    """One tensor on the host, or on another GPU than the others."""
    call, args = CALLS[name]
    for other in (torch.Tensor, OnAnotherGpu):
        if other is OnAnotherGpu and len(args) == 1:
            continue
        with pytest.raises(ValueError, match="must be on one GPU"):
            call(**{**args, arg: args[arg].as_subclass(other)})


def test_the_current_device(monkeypatch):
    """Tensors on one GPU while another is current, or with another's stream."""
    class Library:
        def __getattr__(self, name):
            raise AssertionError(name)

    class Stream:
        device_index, cuda_stream = 1, 0

    monkeypatch.setattr(bsmm, "load", Library)
    monkeypatch.setattr(bsmm, "_CURRENT", [(lambda: 1, lambda device: 0)])
    x = t(4, 32)
    for stream, what in ((None, "current device"), (Stream, "stream")):
        with pytest.raises(ValueError, match=what):
            bsmm._stream_of(x, stream)
