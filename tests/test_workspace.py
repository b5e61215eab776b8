"""Which workspace the binding hands to a call (no GPU needed: the policy
does not look at the device)."""

from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import block_scaled_precision_gemm_amd as bsmm

CPU = torch.device("cpu")


@pytest.fixture(autouse=True)
def _own_cache(monkeypatch):
    """These buffers are on the host: they stay out of the real cache, and
    there is no stream to ask."""
    monkeypatch.setattr(bsmm, "_WS", type(bsmm._WS)())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)


def test_eager_calls_of_a_stream_share_a_buffer():
    a, n = bsmm._buffer(64, CPU, None, 1)
    assert n == 64 and bsmm._buffer(32, CPU, None, 1) == (a, 64)
    b, n = bsmm._buffer(128, CPU, None, 1)
    assert n == 128 and bsmm._buffer(64, CPU, None, 1) == (b, 128)
    assert bsmm._buffer(64, CPU, None, 2)[0] != b
    assert bsmm._buffer(0, CPU, None, 3) == (None, 0)


def test_a_captured_call_has_its_own_buffer(monkeypatch):
    """Nothing that a graph recorded is handed to another call, eager or
    captured, and no cached address is recorded."""
    eager, _ = bsmm._buffer(64, CPU, None, 1)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    a, n = bsmm._buffer(64, CPU, None, 1)
    b, _ = bsmm._buffer(64, CPU, None, 1)
    assert n == 64 and len({int(eager), int(a), int(b)}) == 3
    # alive for as long as the address is held: until the call's launches
    assert a.buffer.data_ptr() == a
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    assert bsmm._buffer(64, CPU, None, 1) == (eager, 64)


def test_threads_have_their_own_buffers():
    """The launches of two threads' calls on one stream may alternate."""
    mine = bsmm._buffer(64, CPU, None, 1)
    with ThreadPoolExecutor(1) as pool:
        def theirs():
            return pool.submit(bsmm._buffer, 64, CPU, None, 1).result()
        other = theirs()
        assert other[0] != mine[0]
        assert theirs() == other and bsmm._buffer(64, CPU, None, 1) == mine


def test_a_given_workspace():
    """Its address and size are passed on, and the cache stays empty."""
    ws = torch.empty(100, dtype=torch.float32)
    for given, want in ((ws, (ws.data_ptr(), 400)), (False, (None, 0))):
        got = bsmm._w4_workspace(given, bsmm.F32, 1, 2048, 2048, 4096, 4096, 128, CPU, None, 1)
        assert got == want and not bsmm._WS.by
    for call in (bsmm.bsmm_w4_mm, bsmm.bsmm_w4_expert_mm, bsmm.bsmm_route_topk):
        assert "workspace" in call.__kwdefaults__
    assert bsmm.bsmm_w4_workspace_bytes(torch.float32, 1, 2048, 2048, 4096, 4096, 128) == \
        3 * 2048 * 4096 * 2
    assert bsmm.bsmm_route_workspace_bytes(100, 64) > 0
