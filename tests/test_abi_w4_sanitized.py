"""The refusals of the 4-bit weight operations and the router against the
library whose host code is built with AddressSanitizer and
UndefinedBehaviorSanitizer."""

import os

from test_abi_sanitized import _run, san_env  # noqa: F401


def test_refusals_under_asan_and_ubsan(san_env):  # noqa: F811
    out = _run(san_env, ["-m", "pytest", "-x", "-q", "-p", "no:cacheprovider",
                         os.path.join("tests", "test_abi_w4.py")])
    assert " passed" in out and " failed" not in out, out[-2000:]
