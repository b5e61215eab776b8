"""The binding's dtype table: when several threads make it, and what it does
not hold (no GPU needed)."""

import threading

import pytest
import torch

import block_scaled_precision_gemm_amd as bsmm


@pytest.mark.parametrize("at", range(1, 9))
def test_another_thread_during_the_first_use(at, monkeypatch):
    """A thread that comes while another makes the table never meets a part
    of it."""
    failed, asked = [], []

    def refusal():
        # gets past the dtypes, and is refused for its group
        try:
            bsmm.bsmm_quant_w4(torch.zeros(2, 64), group=7)
        except ValueError as e:
            if "group" in str(e):
                return
            failed.append(e)
        except Exception as e:
            failed.append(e)
        else:
            failed.append("accepted")

    class Slow:
        """torch, with the other thread's whole call when dtype number ``at`` is
        asked for."""

        def __getattr__(self, name):
            if isinstance(getattr(torch, name), torch.dtype):
                asked.append(name)
            if len(asked) == at:
                asked.append("done")
                monkeypatch.setattr(bsmm, "_torch", lambda: torch)
                t = threading.Thread(target=refusal)
                t.start()
                t.join(30)
            return getattr(torch, name)

    monkeypatch.setattr(bsmm, "_DTYPES", type(bsmm._DTYPES)())
    slow = Slow()
    monkeypatch.setattr(bsmm, "_quant_input", lambda x, name: (x, bsmm.F32))
    monkeypatch.setattr(bsmm, "_torch", lambda: slow)
    refusal()
    assert not failed


@pytest.mark.parametrize("dt", ["torch", None, (), 7, torch.float16])
def test_other_names_are_refused(dt):
    x, w, s = torch.zeros(2, 128), torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 1)
    with pytest.raises(ValueError, match="expected bf16 or fp32"):
        bsmm.bsmm_w4_mm(x, w, s, out_dtype=dt)
    with pytest.raises(ValueError, match="expected bf16 or fp32"):
        bsmm.bsmm_quant_w4(x, scale_dtype=dt)
