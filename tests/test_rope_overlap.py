"""Rotary positions of rows that share memory: refused on the host before anything is enqueued (no GPU)."""
import ctypes

import pytest

import decode_attention_02_gb300 as mfa
from decode_attention_02_gb300 import build

P = ctypes.c_void_p
CONFIG = mfa.MfaRopeConfig(128, 128, 1, (ctypes.c_int32 * 4)(64), 0, 0, 1e4, 1.0)


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return mfa.load_library()


def rows(i, o, si=512, so=512, heads=4):
    return mfa.MfaRopeRows(i, o, si, so, heads)


@pytest.mark.parametrize("q, k", [
    (rows(0x10000, 0x900000), rows(0x20000, 0x900000)),                        # one output for both
    (rows(0x10000, 0x900000), rows(0x20000, 0x900400)),                        # a row on
    (rows(0x10000, 0x20000), rows(0x20000, 0x900000)),                         # q into k's rows
    (rows(0x10000, 0x900000), rows(0x20000, 0x10000)),                         # k into q's
    (rows(0x10000, 0x10000), rows(0x10000, 0x10000)),                          # both in place on the same rows
    (rows(0x10000, 0x10000, 2048, 2048), rows(0x10300, 0x10300, 2048, 2048)),  # columns that overlap by a quarter
    (rows(0x10300, 0x10300, 2048, 2048), rows(0x10000, 0x10000, 2048, 2048)),
    (rows(0x10000, 0x10000, 2048, 2048), rows(0x10c80, 0x10c80, 2048, 2048)),  # into the next row
    (rows(0x10000, 0x10000, 2048, 2048), rows(0x10400, 0x10400, 1024, 1024)),  # other strides
])
def test_rows_that_share_memory_are_refused(lib, q, k):
    for a, b in ((q, k), (k, q)):
        assert lib.mfa_rope_run(CONFIG, P(0x1000), P(0x2000), 8, 0, 0, a, b, None) == mfa.MFA_ERR_INVALID_ARG


def test_rows_that_no_memory_holds_are_refused(lib):
    """2^31 rows 2^40 elements apart: their extent does not wrap around into a small one."""
    far = rows(0x10000, 0x900000, 1 << 40, 1 << 40)
    assert lib.mfa_rope_run(CONFIG, P(0x1000), P(0x2000), 2 ** 31 - 1, 1, 0, far, None, None) == mfa.MFA_ERR_INVALID_ARG
