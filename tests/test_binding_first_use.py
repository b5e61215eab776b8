"""The binding's dtype table when several threads make it (no GPU needed)."""

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

    monkeypatch.setattr(bsmm, "_DTYPES", {})
    slow = Slow()
    monkeypatch.setattr(bsmm, "_quant_input", lambda x, name: (x, bsmm.F32))
    monkeypatch.setattr(bsmm, "_torch", lambda: slow)
    refusal()
    assert not failed
