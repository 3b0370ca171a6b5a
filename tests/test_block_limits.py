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


def gdr(lib, backward, T, B, H, Hk, K, V):
    qkv = (p(1), Hk * K, p(2), Hk * K, p(3), H * V)
    end = (T, B, H, Hk, K, V, F(1.0), 0, None, 0, None)
    if backward:
        return lib.lrs_gdr_bwd(*qkv, p(4), p(5), None, p(6), p(7), None, p(8), Hk * K, p(9), Hk * K, p(10), H * V,
                               p(11), p(12), None, *end)
    return lib.lrs_gdr_fwd(*qkv, p(4), p(5), None, None, p(6), None, p(7), *end)


def test_chunks_of_the_delta_rule(lib):
    """A workgroup of 256 threads a chunk and head forward, of 512 backward: 2^32 threads are too
    many for a launch."""
    from linear_recurrence_scan_diagonal_amd import binding as b
    for backward, most in ((False, 1 << 24), (True, 1 << 23)):
        query = lib.lrs_gdr_bwd_workspace_bytes if backward else lib.lrs_gdr_workspace_bytes
        for B, H, Hk in ((1, 8, 1), (4, 2, 2)):
            T = 64 * (most // 8)
            assert gdr(lib, backward, T, B, H, Hk, 1, 1) == b.LRS_ERR_UNSUPPORTED
            assert query(T, B, H, Hk, 1, 1, 0) == 0
            assert gdr(lib, backward, T - 64, B, H, Hk, 1, 1) == b.LRS_ERR_WORKSPACE
            assert query(T - 64, B, H, Hk, 1, 1, 0) > 0


def test_padded_rows_of_a_state(lib):
    """Kept states have rows of V rounded up to 4, and their chunk's bytes stay below 2^31."""
    from linear_recurrence_scan_diagonal_amd import binding as b
    for backward in (False, True):
        for K, V in ((128, (1 << 29) // 192 // 4 * 4), (64, (1 << 22) - 4), (1, (1 << 23) - 8)):
            if (K + 64) * V < 1 << 29:
                assert gdr(lib, backward, 1, 1, 1, 1, K, V) == b.LRS_ERR_WORKSPACE, (K, V)
            for more in (1, 2, 3, 4):  # the next four
                if (K + 64) * (V + more) < 1 << 29 <= (K + 64) * (V + 4):
                    assert gdr(lib, backward, 1, 1, 1, 1, K, V + more) == b.LRS_ERR_UNSUPPORTED, (K, V + more)
