"""The queries for the kernel of an experts' product and of its weight
gradient, and the rules behind them (no GPU needed)."""

import os
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
    assert wgrad("bf16", True, 32, 4096, 32768, 2048, 4096, aligned=False)[0] == "tile128"
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
