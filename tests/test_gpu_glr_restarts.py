"""What a restart of the gated linear recurrence cuts, and what it does not: values
that are not finite in any of the inputs, at several distances before and after a
restart, in both plans (look-back tiles, and the persistent walk of many channels),
forward and backward, against the plain fp64 form (lm_ref.py).

A value has to be NaN exactly where the plain form's is; the finite ones obey the
bounds of test_gpu_glr.py (1e-5 of 1 + |value|, plus 2^-8 of the value in bf16)."""
import numpy as np
import pytest
import torch

import linear_recurrence_scan_diagonal_amd as lrs
import lm_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = {torch.float32: 1e-5, torch.bfloat16: 2.0 ** -8 + 1e-5}
NAMES = ("grad_zr", "grad_zi", "grad_x", "grad_bias_r", "grad_bias_i", "grad_decay", "grad_h0")
# (T, B, D): a few channels take look-back tiles, more than 2^15 the persistent walk
SIZES = {"tiles": (300, 1, 70), "ragged tiles": (203, 3, 33), "walk": (200, 65, 512),
         "ragged walk": (139, 64, 521)}


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def make(T, B, D, dtype, seed=0, decay=-5.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    parts = [n(T, B, D).to(dtype).to(DEV) for _ in range(3)]
    p = {"bias_r": 0.3 * n(D), "bias_i": 0.3 * n(D), "decay": decay + 0.5 * n(D)}
    s = {"h0": n(B, D), "gh": n(T, B, D).to(dtype), "gl": n(B, D)}
    return parts, {k: v.to(DEV) for k, v in p.items()}, {k: v.to(DEV) for k, v in s.items()}


def check(parts, p, s, reset):
    dtype = parts[0].dtype
    ck = lrs.glr_checkpoints(parts[0])
    h, last = lrs.glr_fwd(*parts, **p, reset=reset, h0=s["h0"], want_h_last=True, checkpoints=ck)
    grads = lrs.glr_bwd(*parts, **p, checkpoints=ck, grad_h=s["gh"], reset=reset,
                        grad_h_last=s["gl"])
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore", over="ignore"):
        ref = R.glr(*(f64(t) for t in parts), f64(p["bias_r"]), f64(p["bias_i"]), f64(p["decay"]), 8.0,
                    reset.cpu().numpy(), f64(s["h0"]), f64(s["gh"]), f64(s["gl"]))
    got = {"h": h, "h_last": last, **dict(zip(NAMES, grads))}
    for name, t in got.items():
        t, want = f64(t), ref[name]
        nan = np.isnan(want)
        assert np.array_equal(np.isnan(t), nan), (name, int(np.isnan(t).sum()), int(nan.sum()))
        own = ref.get("scale_" + name)  # the parameters' gradients: of the sum's absolute terms
        size = 1 + np.abs(want if own is None else own)
        tol = TOL[dtype] if t.ndim == 3 else 1e-5
        off = np.abs(t - want)[~nan] / size[~nan]
        assert off.max(initial=0.0) <= tol, (name, off.max())
    return got, ref


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("where", ["z_r", "z_i", "x"])
def test_nan_stays_in_its_document(size, dtype, where):
    """NaN at 1 to 60 steps before a restart, in the same wave's rows as the restart,
    in an earlier wave's of the same tile, and in an earlier tile; and in a later
    document, whose gradients must not reach the earlier one."""
    T, B, D = SIZES[size]
    parts, p, s = make(T, B, D, dtype, seed=T)
    reset = torch.zeros((T, B), dtype=torch.uint8, device=DEV)
    reset[20] = reset[100] = 1
    reset[T - 3] = 1
    z = parts[["z_r", "z_i", "x"].index(where)]
    b = B - 1
    for d, t in enumerate((19, 17, 10, 4, 99, 96, 80, 40, 21, 101, 125, T - 4, T - 1, T - 2, 20 + 3)):
        z[t, b, 2 * d % D] = float("nan")
    got, ref = check(parts, p, s, reset)
    assert np.isnan(ref["h"]).any() and np.isfinite(ref["h"][20]).all()
    assert np.isfinite(ref["h"][100]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", SIZES)
def test_whole_rows_of_nan(size, dtype):
    """A row that overflowed holds NaN in all three parts."""
    T, B, D = SIZES[size]
    parts, p, s = make(T, B, D, dtype, seed=T + 1)
    reset = torch.zeros((T, B), dtype=torch.uint8, device=DEV)
    reset[20] = reset[90] = reset[130] = 1
    for t, b in ((10, 0), (83, B - 1), (125, B // 2)):
        for z in parts:
            z[t, b] = float("nan")
    check(parts, p, s, reset)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("decay", [2.0, 30.0])
def test_only_a_restart_cuts(size, dtype, decay):
    """A short memory (a = exp(-17 r), and exp(-240 r) that fp32 rounds to 0) lets a
    finite state fade, but a NaN stays to the end of its document, whether the call
    has restarts or not; so does one of the gradient to the document's beginning."""
    T, B, D = SIZES[size]
    parts, p, s = make(T, B, D, dtype, seed=T + 2, decay=decay)
    reset = torch.zeros((T, B), dtype=torch.uint8, device=DEV)
    reset[T - 20] = 1
    parts[2][5, 0, 3] = float("nan")
    parts[0][7, B - 1, 8] = float("nan")
    s["gh"][T - 40, B // 2, 11] = float("nan")
    got, ref = check(parts, p, s, reset)
    assert np.isnan(ref["h"][5:T - 20, 0, 3]).all() and np.isfinite(ref["h"][T - 20:]).all()
    assert np.isnan(ref["grad_x"][:T - 39, B // 2, 11]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", SIZES)
def test_a_restart_does_not_look_at_its_own_gate(size, dtype):
    """At a restart a = 0 and m = 1 whatever z_r is: the same results with a NaN there, and
    a zero gradient."""
    T, B, D = SIZES[size]
    parts, p, s = make(T, B, D, dtype, seed=T + 3)
    reset = torch.zeros((T, B), dtype=torch.uint8, device=DEV)
    reset[0] = reset[33] = reset[64] = reset[T - 1] = 1
    want, _ = check(parts, p, s, reset)
    parts[0][reset != 0] = float("nan")
    ck = lrs.glr_checkpoints(parts[0])
    h, last = lrs.glr_fwd(*parts, **p, reset=reset, h0=s["h0"], want_h_last=True, checkpoints=ck)
    grads = lrs.glr_bwd(*parts, **p, checkpoints=ck, grad_h=s["gh"], reset=reset, grad_h_last=s["gl"])
    for name, t in {"h": h, "h_last": last, **dict(zip(NAMES, grads))}.items():
        assert torch.equal(t, want[name]), name
    assert (grads[0][reset != 0] == 0).all()
