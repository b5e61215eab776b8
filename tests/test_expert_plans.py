"""The queries for the kernel of an experts' product and of its weight
gradient, and the rules behind them (no GPU needed)."""

import os
import random
import re

import pytest

import block_scaled_precision_gemm_amd as bsmm

mm, wgrad = bsmm.bsmm_expert_mm_plan_name, bsmm.bsmm_expert_wgrad_plan_name


def test_product():
    # few rows an expert: straight to registers, if they are aligned
    assert mm("bf16", False, 64, 8, 2048, 4096) == ("rows", 1)
    assert mm("f32", True, 16, 64, 1024, 4096) == ("rows", 1)
    assert mm("bf16", False, 64, 8, 2048, 4096, aligned=False)[0] != "rows"
    assert mm("bf16", False, 64, 8, 2048, 4097)[0] != "rows"
    # many: as high as fills the chip
    assert mm("bf16", False, 64, 32768, 2048, 4096) == ("wide256", 1)
    assert mm("bf16", True, 1, 8192, 8192, 8192) == ("wide256", 1)
    assert {mm("bf16", False, 16, s, 2048, 2048)[0] for s in range(1024, 9000, 64)} == \
        {"wide128", "wide192", "wide256"}
    assert mm("f32", False, 16, 4000, 1024, 2048) == ("tile64", 1)
    # few tiles: ranges of K, no more than the workspace holds
    name, parts = mm("bf16", False, 1, 300, 130, 4096)
    assert name == "wide128" and parts > 1
    assert bsmm.bsmm_expert_mm_workspace_bytes("bf16", False, 1, 300, 130, 4096) == \
        parts * 300 * 130 * 4
    assert mm("bf16", False, 1, 300, 130, 4096, workspace=0)[1] == 1


def test_weight_gradient():
    assert wgrad("bf16", False, 32, 4096, 32768, 2048, 4096) == ("wide256", 1)
    assert wgrad("bf16", True, 32, 4096, 32768, 2048, 4096) == ("restored", 1)
    assert wgrad("bf16", True, 32, 4096, 32768, 2048, 4096, workspace=0) == ("tile128", 1)
    assert wgrad("bf16", True, 32, 4096, 32768, 2048, 4096, x_aligned=False)[0] == "tile128"
    assert wgrad("f32", True, 32, 4096, 32768, 2048, 4096)[0].startswith("tile")
    assert wgrad("f32", False, 6, 333, 666, 1001, 515) == ("tile64", 1)
    assert wgrad("bf16", False, 1, 9000, 9000, 64, 72)[1] > 1
    assert wgrad("bf16", False, 1, 9000, 9000, 64, 72, workspace=0)[1] == 1


@pytest.mark.parametrize("bad", [(0, 9, 9, 9), (1025, 9, 9, 9), (1, 0, 9, 9), (1, 2**31, 9, 9),
                                 (1, 9, -1, 9), (1, 9, 9, 0)])
def test_sizes_without_a_kernel(bad):
    E, S, N, K = bad
    assert mm("f32", False, *bad) is None and mm("bf16", True, *bad) is None
    assert wgrad("f32", False, E, S, S, N, K) is None
    assert wgrad("bf16", True, 1, 9, 9, 9, 40) is None


@pytest.mark.parametrize("value", ["0", "", "100000"])
def test_the_environment_changes_no_plan(value, monkeypatch):
    sizes = [("bf16", False, 64, 8, 2048, 4096), ("bf16", False, 64, 8168, 2048, 4096),
             ("f32", True, 16, 64, 1024, 4096), ("f32", False, 16, 900, 1024, 2048)]
    before = [mm(*c) for c in sizes]
    monkeypatch.setenv("FEW", value)
    assert [mm(*c) for c in sizes] == before


def test_every_variable_has_the_librarys_name():
    csrc = os.path.join(os.path.dirname(bsmm.__file__), "csrc")
    for name in sorted(os.listdir(csrc)):
        with open(os.path.join(csrc, name)) as f:
            for argument in re.findall(r"getenv\(([^)]*)\)", f.read()):
                assert argument.startswith('"BSMM_'), (name, argument)


def random_sizes(n, seed):
    rng = random.Random(seed)
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))  # noqa: E731
    for _ in range(n):
        N, K = log(16, 8192), log(16, 8192)
        if rng.random() < 0.6:
            N, K = max(32, N // 32 * 32), max(32, K // 32 * 32)
        yield rng.random() < 0.5, log(1, 64), log(1, 30000), N, K


NAMED = [(True, 1, 804, 2872, 3136), (True, 4, 1222, 1840, 2688), (True, 15, 11712, 72, 1760)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_larger_workspace_changes_nothing(dt):
    """The order of the sums follows from the call alone: with the bytes that
    the query gives the plan is that of any larger workspace, such as one that
    other calls have left."""
    for back, E, S, N, K in NAMED + list(random_sizes(4000, 1)):
        for rows in (True, False):
            same = {mm(dt, back, E, S, N, K, aligned=rows, workspace=room)
                    for room in (None, 2**27 + 12345, 2**28, 2**40)
                    if room is None or
                    room >= bsmm.bsmm_expert_mm_workspace_bytes(dt, back, E, S, N, K)}
            assert len(same) == 1, (back, E, S, N, K, rows, same)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("checkpoint", [False, True])
def test_a_larger_workspace_changes_no_gradient(checkpoint, dt):
    for second, E, S, N, K in random_sizes(4000, 2):
        K = max(32, K // 32 * 32) if checkpoint else K
        Rx = max(1, S // 4) if second else S
        need = bsmm.bsmm_expert_wgrad_workspace_bytes(dt, checkpoint, E, Rx, S, N, K)
        for odt in ("bf16", "f32"):
            for rows in ((True, True), (True, False), (False, True), (False, False)):
                same = {wgrad(dt, checkpoint, E, Rx, S, N, K, out_dtype=odt, workspace=room,
                              dy_aligned=rows[0], x_aligned=rows[1])
                        for room in (None, 2**27 + 12345, 2**28, 2**40)
                        if room is None or room >= need}
                assert len(same) == 1, (E, Rx, S, N, K, odt, rows, same)


def test_a_smaller_workspace_is_enough_for_its_plan():
    rng = random.Random(3)
    for back, E, S, N, K in NAMED + list(random_sizes(2000, 4)):
        need = bsmm.bsmm_expert_mm_workspace_bytes("bf16", back, E, S, N, K)
        for room in (0, need // 2, rng.randint(0, need)):
            parts = mm("bf16", back, E, S, N, K, workspace=room)[1]
            assert parts == 1 or parts * S * N * 4 <= room
        K = max(32, K // 32 * 32)
        values = S * K * 2
        need = bsmm.bsmm_expert_wgrad_workspace_bytes("bf16", True, E, S, S, N, K)
        for room in (0, need // 2, values - 1, values, rng.randint(0, need)):
            name, parts = wgrad("bf16", True, E, S, S, N, K, workspace=room)
            used = (values if name == "restored" else 0) + \
                (parts * E * N * K * 4 if parts > 1 else 0)
            assert used <= room
