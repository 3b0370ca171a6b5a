"""include/lrs_block.h without a GPU: every declared function is exported and bound, and
validation and workspace queries behave as the header states.  No call here reaches a
HIP runtime function."""
import ctypes
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "linear_recurrence_scan_diagonal_amd", "liblrs.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="liblrs.so not built")
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    from linear_recurrence_scan_diagonal_amd import block
    return block.load()


def q(n):
    return ctypes.c_void_p(0x1000000 * n)  # never dereferenced: every call below is refused


def test_declared_exported_and_bound(lib):
    from linear_recurrence_scan_diagonal_amd import block
    text = open(os.path.join(ROOT, "include", "lrs_block.h")).read()
    names = sorted(set(re.findall(r"LRS_API\s+[\w\s\*]*?\b(lrs_\w+)\s*\(", text)))
    assert names == sorted(block.EXPORTS) and len(names) == 12
    raw = ctypes.CDLL(LIB)
    for n in names:
        assert hasattr(raw, n) and getattr(lib, n).argtypes is not None


def test_public_names():
    import linear_recurrence_scan_diagonal_amd as lrs
    for n in ("gdr_checkpoints", "gdr_fwd", "gdr_bwd", "gdr_step", "rmsnorm_fwd", "rmsnorm_fwd_fp8",
              "rmsnorm_bwd", "logprobs_fwd", "logprobs_bwd"):
        assert n in lrs.__all__ and callable(getattr(lrs, n))


def test_load_sets_the_prototypes_of_every_function():
    """In a process that has called nothing yet."""
    code = ("import linear_recurrence_scan_diagonal_amd as lrs\n"
            "lib = lrs.load()\n"
            "from linear_recurrence_scan_diagonal_amd import binding, block, lm\n"
            "print(all(getattr(lib, n).argtypes is not None for n in binding.EXPORTS + lm.EXPORTS + block.EXPORTS))\n"
            "print(lib.lrs_gdr_bwd_workspace_bytes(65536, 16, 16, 16, 128, 128, 1))\n")
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True, capture_output=True, text=True)
    prototypes, nbytes = out.stdout.split()
    assert prototypes == "True" and int(nbytes) > 2 ** 33


def test_queries(lib):
    rows = lib.lrs_gdr_checkpoint_rows
    assert [rows(t) for t in (-3, 0, 1, 64, 65, 2048)] == [0, 0, 1, 1, 2, 32]
    # shared heads: the operands of q and k once; the backward keeps a gradient for each as well
    fwd = lib.lrs_gdr_workspace_bytes
    assert fwd(100, 2, 4, 2, 64, 64, 1) < fwd(100, 2, 4, 4, 64, 64, 1)
    for query in (lib.lrs_gdr_workspace_bytes, lib.lrs_gdr_bwd_workspace_bytes):
        assert query(0, 4, 4, 4, 64, 64, 1) == 0 and query(4, 0, 4, 4, 64, 64, 1) == 0
        assert query(4, 4, 4, 3, 64, 64, 1) == 0  # heads that cannot be shared
        assert query(4, 4, 4, 4, 129, 64, 1) == 0 and query(4, 4, 4, 4, 0, 64, 1) == 0
        assert query(4, 4, 4, 4, 64, 64, 7) == 0 and query(-1, 4, 4, 4, 64, 64, 1) == 0
        assert query(1 << 40, 1 << 40, 4, 4, 64, 64, 1) == 0
        assert query(100, 2, 4, 4, 64, 64, 0) >= query(100, 2, 4, 4, 64, 64, 1) > 0
    assert lib.lrs_rmsnorm_bwd_workspace_bytes(0, 8) == 0
    assert lib.lrs_rmsnorm_bwd_workspace_bytes(100, 64) >= 25 * 64 * 4


def test_gdr_refusals(lib):
    from linear_recurrence_scan_diagonal_amd import binding as b
    bad, ws, not_supported = b.LRS_ERR_INVALID_ARG, b.LRS_ERR_WORKSPACE, b.LRS_ERR_UNSUPPORTED

    def fwd(q_=q(1), ldq=32, k=q(2), ldk=32, v=q(3), ldv=64, g=q(4), be=q(5), r=None, s0=None, o=q(6), s=None,
            ck=None, T=4, B=2, H=4, Hk=2, K=16, V=16, scale=1.0, io=0):
        return lib.lrs_gdr_fwd(q_, ldq, k, ldk, v, ldv, g, be, r, s0, o, s, ck, T, B, H, Hk, K, V, F(scale), io,
                               None, 0, None)
    assert fwd() == ws
    for name in ("q_", "k", "v", "g", "be", "o"):
        assert fwd(**{name: None}) == bad, name
    assert fwd(ldq=31) == bad and fwd(ldk=31) == bad and fwd(ldv=63) == bad
    assert fwd(H=3) == bad and fwd(Hk=0) == bad and fwd(K=0) == bad and fwd(V=0) == bad and fwd(T=-1) == bad
    assert fwd(io=2) == bad and fwd(scale=float("inf")) == bad and fwd(scale=float("nan")) == bad
    assert fwd(o=q(3)) == bad and fwd(ck=q(6)) == bad and fwd(s=q(1)) == bad
    assert fwd(s0=q(7), s=q(7)) == ws  # the state in place
    assert fwd(s0=q(7), s=ctypes.c_void_p(0x7000004)) == bad
    assert fwd(q_=ctypes.c_void_p(0x1000002)) == bad and fwd(q_=ctypes.c_void_p(0x1000002), io=1) == ws
    assert fwd(K=129, ldq=258, ldk=258) == not_supported
    assert fwd(T=1 << 24, H=1024, Hk=2, V=16, ldv=1024 * 16, q_=q(1 << 8), k=q(1 << 16), v=q(1 << 20), o=q(1 << 21),
               g=q(1 << 22), be=q(1 << 22 | 1 << 18)) == not_supported
    assert fwd(T=0) == b.LRS_OK and fwd(B=0) == b.LRS_OK and fwd(B=0, s=q(9)) == b.LRS_OK

    def bwd(gq=q(11), ldgq=32, gk=q(12), ldgk=32, gv=q(13), ldgv=64, ck=q(8), go=q(9), gs=None, gg=q(14), gb=q(15),
            gs0=None, T=4):
        return lib.lrs_gdr_bwd(q(1), 32, q(2), 32, q(3), 64, q(4), q(5), None, ck, go, gs, gq, ldgq, gk, ldgk, gv,
                               ldgv, gg, gb, gs0, T, 2, 4, 2, 16, 16, F(1.0), 0, None, 0, None)
    assert bwd() == ws
    for name in ("gq", "gk", "gv", "ck", "go", "gg", "gb"):
        assert bwd(**{name: None}) == bad, name
    assert bwd(gq=q(12)) == bad and bwd(gv=q(1)) == bad and bwd(gg=q(15)) == bad and bwd(gb=q(9)) == bad
    assert bwd(ldgq=31) == bad and bwd(gs=q(16), gs0=q(16)) == ws and bwd(gs0=q(8)) == bad
    assert bwd(T=0) == b.LRS_OK
    # slices of one gradient (of 32, 32 and 64 elements) interleave without sharing an element
    base = 0x21000000
    at = lambda n: ctypes.c_void_p(base + 4 * n)  # noqa: E731
    three = dict(gq=at(0), gk=at(32), gv=at(64), ldgq=128, ldgk=128, ldgv=128)
    assert bwd(**three) == ws
    assert bwd(**{**three, "gk": at(31)}) == bad and bwd(**{**three, "gv": at(63)}) == bad
    assert bwd(**{**three, "gv": at(65)}) == bad  # its end is the next row's first element of q
    assert bwd(**{**three, "gk": at(33)}) == bad and bwd(**{**three, "ldgv": 130}) == bad

    def step(slots=q(8), state=q(9), S=4, B=2, o=q(10), K=16, ld=32):
        return lib.lrs_gdr_step(q(1), ld, q(2), ld, q(3), 64, q(4), q(5), slots, state, o, B, 4, 2, K, 16, S, F(1.0),
                                0, None)
    assert step(state=None) == bad and step(slots=None, S=1) == bad and step(S=-1) == bad
    assert step(o=q(9)) == bad and step(ld=31) == bad and step(K=129, ld=300) == not_supported
    assert step(B=0) == b.LRS_OK


def test_rmsnorm_refusals(lib):
    from linear_recurrence_scan_diagonal_amd import binding as b
    bad = b.LRS_ERR_INVALID_ARG

    def fwd(x=q(1), res=None, y=q(4), s=None, rstd=None, R=2, D=8, eps=1e-5, io=0):
        return lib.lrs_rmsnorm_fwd(x, res, q(2), y, s, rstd, R, D, F(eps), io, None)
    assert fwd(x=None) == bad and fwd(y=None) == bad and fwd(eps=-1.0) == bad and fwd(eps=float("nan")) == bad
    assert fwd(res=q(5)) == bad and fwd(s=q(5)) == bad  # residual and sum go together
    assert fwd(y=q(1)) == bad and fwd(rstd=q(4)) == bad and fwd(io=5) == bad and fwd(R=-1) == bad
    assert fwd(res=q(5), s=q(4)) == bad and fwd(R=0) == b.LRS_OK and fwd(x=q(1 << 12), y=q(1 << 16), R=1 << 23, D=2000) == b.LRS_ERR_UNSUPPORTED

    def fp8(scales=q(5), group=128, y=q(4), R=2):
        return lib.lrs_rmsnorm_fwd_fp8(q(1), None, q(2), y, scales, None, R, 8, group, F(1e-5), 0, None)
    assert fp8(scales=None) == bad and fp8(group=64) == bad and fp8(group=-1) == bad and fp8(y=q(1)) == bad
    assert fp8(scales=q(4)) == bad and fp8(scales=q(1)) == bad and fp8(R=0) == b.LRS_OK
    assert fp8(scales=ctypes.c_void_p(0x5000002)) == bad

    def bwd(s=q(1), gy=q(5), gsum=None, gx=q(6), gg=q(7)):
        return lib.lrs_rmsnorm_bwd(s, q(2), q(4), gy, gsum, gx, gg, 2, 8, 0, None, 0, None)
    assert bwd(s=None) == bad and bwd(gx=q(1)) == bad and bwd(gg=q(6)) == bad and bwd(gg=q(5), gx=q(5)) == bad
    assert bwd() == b.LRS_ERR_WORKSPACE and bwd(gx=q(5)) == b.LRS_ERR_WORKSPACE
    assert bwd(gsum=q(8), gx=q(8)) == b.LRS_ERR_WORKSPACE


def test_logprobs_refusals(lib):
    from linear_recurrence_scan_diagonal_amd import binding as b
    bad = b.LRS_ERR_INVALID_ARG

    def fwd(x=q(1), ld=8, t=q(2), lp=q(3), en=q(4), lse=q(5), ids=q(6), tops=q(7), N=2, V=8, top=3, io=0):
        return lib.lrs_logprobs_fwd(x, ld, t, lp, en, lse, ids, tops, N, V, top, io, None)
    for name in ("x", "t", "lp", "en", "lse", "ids", "tops"):
        assert fwd(**{name: None}) == bad, name
    assert fwd(ld=7) == bad and fwd(top=9) == bad and fwd(top=-1) == bad and fwd(top=65, V=100, ld=100) == bad
    assert fwd(V=0) == bad and fwd(N=-1) == bad and fwd(io=3) == bad and fwd(lp=q(4)) == bad and fwd(tops=q(1)) == bad
    assert fwd(t=ctypes.c_void_p(0x2000004)) == bad and fwd(N=0) == b.LRS_OK
    assert fwd(V=1 << 24, ld=1 << 24) == b.LRS_ERR_UNSUPPORTED

    def bwd(x=q(1), ld=8, lse=q(3), en=q(4), gl=q(5), ge=q(6), g=q(7), ldg=8, N=2):
        return lib.lrs_logprobs_bwd(x, ld, q(2), lse, en, gl, ge, g, ldg, N, 8, 0, None)
    for name in ("x", "lse", "en", "gl", "g"):
        assert bwd(**{name: None}) == bad, name
    assert bwd(ld=7) == bad and bwd(ldg=7) == bad and bwd(g=q(3)) == bad and bwd(g=q(1), ldg=9) == bad
    assert bwd(g=ctypes.c_void_p(0x1000004)) == bad and bwd(N=0) == b.LRS_OK
