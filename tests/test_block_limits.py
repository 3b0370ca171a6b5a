"""The largest sizes of include/lrs_block.h, without a GPU: one size is taken (a call without a
workspace says so) and the next is refused before any launch."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "linear_recurrence_scan_diagonal_amd", "liblrs.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="liblrs.so not built")
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    from linear_recurrence_scan_diagonal_amd import block
    return block.load()


def p(n):
    return ctypes.c_void_p(n << 44)  # arrays far from each other; never dereferenced


def test_rows_of_logits(lib):
    from linear_recurrence_scan_diagonal_amd import binding as b
    for N, V in ((1 << 24, 2), (2, 1 << 24)):
        assert lib.lrs_logprobs_fwd(p(1), V, p(2), p(3), p(4), p(5), p(6), p(7), N, V, 1, 0, None) == b.LRS_ERR_UNSUPPORTED
        assert lib.lrs_logprobs_bwd(p(1), V, p(2), p(3), p(4), p(5), p(6), p(7), V, N, V, 0, None) == b.LRS_ERR_UNSUPPORTED
