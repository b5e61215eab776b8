"""The query for the kernel of a 4-bit product, and the kernels that the
products' tests name for their sizes (no GPU needed)."""

import pytest

import block_scaled_precision_gemm_amd as bsmm

name = bsmm.bsmm_w4_plan_name


def test_names():
    assert name("bf16", False, 1, 1, 1, 5120, 8192, 128) == "rows4"
    assert name("bf16", False, 1, 5, 5, 5120, 8192, 128) == "rows16"
    assert name("bf16", False, 1, 17, 17, 5120, 8192, 128) == "rows32"
    assert name("f32", False, 1, 17, 17, 5120, 8192, 128) == "rows16"
    assert name("bf16", False, 1, 2047, 2047, 5120, 8192, 128) in ("tile128", "tile256")
    # an expert's average of 2 rows and above
    assert name("bf16", True, 64, 16, 128, 2048, 4096, 128) == "rows4"
    assert name("bf16", True, 64, 17, 129, 2048, 4096, 128) == "rows16"
    # routed calls never take 256 rows
    assert {name("bf16", True, 4, m, m, 5120, 8192, 128) for m in range(200, 9000, 77)} <= \
        {"rows32", "tile128"}


@pytest.mark.parametrize("bad", [(0, 9, 9, 9, 64, 32), (1025, 9, 9, 9, 64, 32),
                                 (1, 0, 9, 9, 64, 32), (1, 9, -1, 9, 64, 32),
                                 (1, 9, 9, 2**31, 64, 32), (1, 9, 9, 9, 0, 32),
                                 (1, 9, 9, 9, 96, 64), (1, 9, 9, 9, 64, 16)])
def test_sizes_without_a_kernel(bad):
    assert name("f32", False, *bad) is None and name("bf16", True, *bad) is None


def test_the_workspace_goes_with_the_tiles():
    for m in (13, 40, 300, 1300, 2047):
        for g in (32, 64, 128):
            for routed, e in ((False, 1), (True, 8)):
                tiled = name("f32", routed, e, m, m, 2100, 1152, g).startswith("tile")
                need = bsmm.bsmm_w4_workspace_bytes("f32", e, m, m, 2100, 1152, g)
                assert need == (3 * m * 1152 * 2 if tiled else 0)
