"""include/lrs_lm.h without a GPU: every declared function is exported and bound,
and validation and workspace queries behave as the header states.  No call here
reaches a HIP runtime function."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "linear_recurrence_scan_diagonal_amd", "liblrs.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="liblrs.so not built")
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    from linear_recurrence_scan_diagonal_amd import lm
    return lm.load()


def q(n):
    return ctypes.c_void_p(0x1000000 * n)  # never dereferenced: every call below is refused


def test_declared_exported_and_bound(lib):
    from linear_recurrence_scan_diagonal_amd import lm
    text = open(os.path.join(ROOT, "include", "lrs_lm.h")).read()
    names = sorted(set(re.findall(r"LRS_API\s+[\w\s\*]*?\b(lrs_\w+)\s*\(", text)))
    assert names == sorted(lm.EXPORTS) and len(names) == 13
    raw = ctypes.CDLL(LIB)
    for n in names:
        assert hasattr(raw, n) and getattr(lib, n).argtypes is not None


def test_public_names():
    import linear_recurrence_scan_diagonal_amd as lrs
    for n in ("glr_checkpoints", "glr_fwd", "glr_bwd", "glr_step", "layernorm_fwd", "layernorm_bwd",
              "linear_ce_fwd", "linear_ce_bwd", "linear_ce_fwd_bwd"):
        assert n in lrs.__all__ and callable(getattr(lrs, n))


def test_queries(lib):
    rows = lib.lrs_glr_checkpoint_rows
    assert [rows(t) for t in (-3, 0, 1, 64, 65, 2048)] == [0, 0, 1, 1, 2, 32]
    assert lib.lrs_glr_workspace_bytes(16, 4, 8) == 0
    assert lib.lrs_glr_workspace_bytes(2048, 4, 512) >= 4 * 512 * 32 * 8
    assert lib.lrs_glr_workspace_bytes(-1, 1, 1) == 0 and lib.lrs_glr_bwd_workspace_bytes(1, -1, 1) == 0
    assert lib.lrs_glr_workspace_bytes(1 << 40, 1 << 40, 2) == 0
    assert lib.lrs_glr_bwd_workspace_bytes(128, 4, 512) >= 3 * 2 * 4 * 512 * 4
    assert lib.lrs_layernorm_bwd_workspace_bytes(0, 8) == 0
    assert lib.lrs_layernorm_bwd_workspace_bytes(100, 64) >= 2 * 25 * 64 * 4
    assert lib.lrs_linear_ce_workspace_bytes(0, 8, 8, 1, 1) == 0
    assert lib.lrs_linear_ce_workspace_bytes(8, 0, 8, 1, 1) == 0
    assert lib.lrs_linear_ce_workspace_bytes(8, 8, 8, 7, 0) == 0
    assert lib.lrs_linear_ce_workspace_bytes(1 << 21, 8, 8, 1, 1) == 0
    # G is made in pieces of the rows: what a call needs beyond copies of its
    # operands and fp32 sums for w's gradient stays bounded
    n, d = 1000000, 64
    for v in (100000, 1000000):
        need = lib.lrs_linear_ce_workspace_bytes(n, v, d, 1, 1)
        assert need < 2 ** 31 + 2 * (n + v) * d * 2 + 16 * v * d * 4 and need < n * v * 2
    assert lib.lrs_linear_ce_workspace_bytes(n, v, d, 1, 0) < need


def test_glr_refusals(lib):
    from linear_recurrence_scan_diagonal_amd import binding as b
    bad, ws = b.LRS_ERR_INVALID_ARG, b.LRS_ERR_WORKSPACE

    def fwd(zr=q(1), zi=q(2), x=q(3), ld=8, h=q(7), hl=None, ck=None, T=4, B=2, D=8, c=8.0, io=0):
        return lib.lrs_glr_fwd(zr, zi, x, ld, q(4), q(5), q(6), None, None, h, hl, ck, T, B, D, F(c),
                               io, None, 0, None)
    assert fwd(zr=None) == bad and fwd(h=None) == bad and fwd(ld=7) == bad and fwd(io=2) == bad
    assert fwd(T=-1) == bad and fwd(c=0.0) == bad and fwd(c=float("nan")) == bad
    assert fwd(c=float("inf")) == bad and fwd(h=q(3)) == bad and fwd(ck=q(7)) == bad
    assert fwd(x=ctypes.c_void_p(0x3000002)) == bad
    assert fwd(T=1000) == ws  # several time tiles need look-back state
    assert fwd(T=0) == b.LRS_OK and fwd(B=0) == b.LRS_OK
    assert fwd(B=1 << 20, D=1 << 12, ld=1 << 12, T=1, zr=q(1 << 12), zi=q(2 << 12), x=q(3 << 12),
               h=q(4 << 12)) == b.LRS_ERR_UNSUPPORTED

    def bwd(gr=q(11), gi=q(12), gx=q(13), ldg=8, ck=q(8), T=4):
        return lib.lrs_glr_bwd(q(1), q(2), q(3), 8, q(4), q(5), q(6), None, ck, q(9), None, gr, gi,
                               gx, ldg, q(14), q(15), q(16), q(17), T, 2, 8, F(8.0), 0, None, 0, None)
    assert bwd(ck=None) == bad and bwd(gr=q(12)) == bad and bwd(ldg=4) == bad and bwd(gx=q(1)) == bad
    assert bwd() == ws
    # slices of one gradient interleave without sharing an element; shifted ones do share
    base = 0x21000000
    three = [ctypes.c_void_p(base + 32 * k) for k in range(3)]
    assert bwd(*three, ldg=24) == ws
    three[2] = ctypes.c_void_p(base + 32 * 2 + 4)
    assert bwd(*three, ldg=24) == bad

    def step(slots=q(8), state=q(9), S=4, B=2, h=q(10)):
        return lib.lrs_glr_step(q(1), q(2), q(3), 8, q(4), q(5), q(6), slots, state, h, B, 8, S,
                                F(8.0), 0, None)
    assert step(state=None) == bad and step(slots=None, S=1) == bad and step(S=-1) == bad
    assert step(h=q(9)) == bad and step(B=0) == b.LRS_OK


def test_layernorm_refusals(lib):
    from linear_recurrence_scan_diagonal_amd import binding as b
    bad = b.LRS_ERR_INVALID_ARG

    def fwd(x=q(1), res=None, y=q(4), s=None, mean=None, rstd=None, R=2, D=8, eps=1e-5, io=0):
        return lib.lrs_layernorm_fwd(x, res, q(2), q(3), y, s, mean, rstd, R, D, F(eps), io, None)
    assert fwd(x=None) == bad and fwd(eps=-1.0) == bad and fwd(eps=float("nan")) == bad
    assert fwd(res=q(5)) == bad and fwd(s=q(5)) == bad  # residual and sum go together
    assert fwd(mean=q(6)) == bad and fwd(y=q(1)) == bad and fwd(io=5) == bad and fwd(R=-1) == bad
    assert fwd(res=q(5), s=q(4)) == bad and fwd(R=0) == b.LRS_OK

    def bwd(s=q(1), gy=q(5), gsum=None, gx=q(6), gg=q(7)):
        return lib.lrs_layernorm_bwd(s, q(2), q(3), q(4), gy, gsum, gx, gg, None, 2, 8, 0, None, 0,
                                     None)
    assert bwd(s=None) == bad and bwd(gx=q(1)) == bad and bwd(gg=q(6)) == bad
    assert bwd() == b.LRS_ERR_WORKSPACE and bwd(gx=q(5)) == b.LRS_ERR_WORKSPACE
    assert bwd(gsum=q(8), gx=q(8)) == b.LRS_ERR_WORKSPACE


def test_linear_ce_refusals(lib):
    from linear_recurrence_scan_diagonal_amd import binding as b
    bad = b.LRS_ERR_INVALID_ARG

    def both(x=q(1), w=q(2), t=q(3), gl=q(4), loss=q(5), lse=q(6), gx=q(7), gw=q(8), N=4, V=8, D=8,
             io=0):
        return lib.lrs_linear_ce_fwd_bwd(x, w, t, gl, loss, lse, gx, gw, N, V, D, io, None, 0, None)
    assert both(x=None) == bad and both(gl=None) == bad and both(V=0) == bad and both(D=0) == bad
    assert both(N=-1) == bad and both(io=3) == bad and both(gx=q(1)) == bad and both(gw=q(7)) == bad
    assert both(lse=q(5)) == bad and both(t=ctypes.c_void_p(0x3000004)) == bad
    assert both() == b.LRS_ERR_WORKSPACE and both(V=1 << 21) == b.LRS_ERR_UNSUPPORTED
    assert lib.lrs_linear_ce_fwd(None, None, None, None, None, 0, 8, 8, 0, None, 0, None) == b.LRS_OK
    # the backward reads lse: it may not be written over
    assert lib.lrs_linear_ce_bwd(q(1), q(2), q(3), q(6), q(4), q(7), q(6), 4, 8, 8, 0, None, 0,
                                 None) == bad
