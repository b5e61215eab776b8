"""4-bit products whose launch would need 2^32 threads, of which the runtime
runs as many as the low 32 bits say: refused, before any HIP call and so
without a GPU (see test_abi_w4.py)."""

import pytest

from test_abi_w4 import UNSUP, experts, mm


@pytest.mark.parametrize("N", [2**30, 2**31 - 1])
def test_columns_of_few_rows(N):
    assert mm(M=1, N=N, K=64, ldx=64, ldw=32, s_n=1, z_n=1, ldo=N) == UNSUP
    assert experts(E=1, R=1, S=1, per=1, N=N, K=64, ldx=64, ldw=32, s_n=1, z_n=1, ldo=N) == UNSUP


def test_tiles_of_many_rows():
    assert mm(M=2**24, N=2**14, K=64, ldx=64, ldw=32, s_n=1, z_n=1, ldo=2**14) == UNSUP
