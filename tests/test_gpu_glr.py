"""Gated linear recurrence on the GPU against the plain fp64 form (lm_ref.py).

Bounds.  An fp32 result carries some tens of roundings of 6e-8 of the values it
is made of: 1e-5 of 1 + |value|, the library's bar.  A bf16 result adds half a
unit in its last place, 2^-8 of the value at most.  The parameters' gradients
are sums over time and batch in fp32 (64 steps) and fp64 (the rest): 1e-5 of the
sum of the absolute terms."""
import numpy as np
import pytest
import torch

import linear_recurrence_scan_diagonal_amd as lrs
import lm_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = {torch.float32: 1e-5, torch.bfloat16: 2.0 ** -8 + 1e-5}


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def make(T, B, D, dtype, seed=0, packed=True, restart=0.0, spread=1.0):
    """Inputs as z_r, z_i, x (slices of one projection if packed) and parameters."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    z = (spread * n(T, B, 3 * D)).to(dtype).to(DEV)
    parts = [z[..., :D], z[..., D:2 * D], z[..., 2 * D:]]
    if not packed:
        parts = [p.contiguous() for p in parts]
    sp = -torch.log(0.9 + 0.0999 * torch.rand(D, generator=g)) / 8.0
    p = dict(bias_r=0.3 * n(D), bias_i=0.3 * n(D), decay=torch.log(torch.expm1(sp)))
    s = dict(h0=n(B, D), gh=n(T, B, D).to(dtype), gl=n(B, D),
             reset=(torch.rand(T, B, generator=g) < restart).to(torch.uint8) if restart else None)
    return parts, {k: v.to(DEV) for k, v in p.items()}, \
        {k: None if v is None else v.to(DEV) for k, v in s.items()}


def reference(parts, p, s, c=8.0, grad=True):
    return R.glr(*(f64(t) for t in parts), f64(p["bias_r"]), f64(p["bias_i"]), f64(p["decay"]), c,
                 None if s["reset"] is None else s["reset"].cpu().numpy(),
                 None if s["h0"] is None else f64(s["h0"]), f64(s["gh"]) if grad else None,
                 None if s["gl"] is None else f64(s["gl"]))


def close(name, got, ref, tol, scale=None):
    got = f64(got)
    assert got.shape == ref.shape, name
    off = np.abs(got - ref) / (1.0 + (np.abs(ref) if scale is None else scale))
    assert np.all(np.isfinite(got)) and (off.size == 0 or off.max() <= tol), (name, off.max())


def check(parts, p, s, c=8.0):
    dtype = parts[0].dtype
    ck = lrs.glr_checkpoints(parts[0])
    h, hl = lrs.glr_fwd(*parts, **p, c=c, reset=s["reset"], h0=s["h0"], want_h_last=True,
                        checkpoints=ck)
    gz = lrs.glr_bwd(*parts, **p, checkpoints=ck, grad_h=s["gh"], c=c, reset=s["reset"],
                     grad_h_last=s["gl"])
    torch.cuda.synchronize()
    ref = reference(parts, p, s, c)
    close("h", h, ref["h"], TOL[dtype])
    close("h_last", hl, ref["h_last"], 1e-5)
    for name, t in zip(("grad_zr", "grad_zi", "grad_x"), gz[:3]):
        close(name, t, ref[name], TOL[dtype])
    for name, t in zip(("grad_bias_r", "grad_bias_i", "grad_decay"), gz[3:6]):
        close(name, t, ref[name], 1e-5, ref["scale_" + name])
    close("grad_h0", gz[6], ref["grad_h0"], 1e-5)
    return h, hl, gz


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,B,D", [
    (1, 1, 1), (1, 3, 5), (2, 1, 128), (63, 2, 64), (64, 1, 130), (65, 3, 37), (129, 2, 256),
    (700, 1, 33), (1024, 2, 128), (640, 5, 129)])
@pytest.mark.parametrize("restart", [0.0, 0.05])
def test_parity(T, B, D, dtype, restart):
    check(*make(T, B, D, dtype, seed=T + D, restart=restart))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_channels(dtype):
    """Enough channel blocks to fill the GPU by themselves, whole and ragged tiles."""
    check(*make(200, 33, 1024, dtype, seed=5))
    check(*make(131, 64, 520, dtype, seed=6, restart=0.03))


def test_contiguous_and_sliced_inputs_agree():
    a = make(150, 2, 96, torch.bfloat16, packed=True, restart=0.02)
    b = make(150, 2, 96, torch.bfloat16, packed=False, restart=0.02)
    ra, rb = check(*a), check(*b)
    assert torch.equal(ra[0], rb[0]) and all(torch.equal(u, v) for u, v in zip(ra[2], rb[2]))


def test_gradients_into_slices_and_misaligned_views():
    parts, p, s = make(130, 3, 62, torch.bfloat16, restart=0.02)
    ck = lrs.glr_checkpoints(parts[0])
    lrs.glr_fwd(*parts, **p, checkpoints=ck, reset=s["reset"], h0=s["h0"])
    want = lrs.glr_bwd(*parts, **p, checkpoints=ck, grad_h=s["gh"], reset=s["reset"])
    gz = torch.full((130, 3, 3 * 62), 7.0, dtype=torch.bfloat16, device=DEV)
    lrs.glr_bwd(*parts, **p, checkpoints=ck, grad_h=s["gh"], reset=s["reset"],
                grad_z=(gz[..., :62], gz[..., 62:124], gz[..., 124:]))
    assert all(torch.equal(gz[..., 62 * k:62 * k + 62], want[k]) for k in range(3))
    # one element past an aligned start, odd pitch: the element-wise path, same bits
    wide = torch.zeros((130, 3, 3 * 62 + 3), dtype=torch.bfloat16, device=DEV)
    moved = []
    for k in range(3):
        v = wide[..., 1 + 62 * k:63 + 62 * k]
        v.copy_(parts[k])
        moved.append(v)
    h = lrs.glr_fwd(*moved, **p, reset=s["reset"], h0=s["h0"])
    assert torch.equal(h, lrs.glr_fwd(*parts, **p, reset=s["reset"], h0=s["h0"]))


def test_optional_arguments():
    parts, p, s = make(100, 2, 40, torch.float32)
    s["h0"] = s["gl"] = None
    check(parts, p, s)
    check(parts, p, s, c=2.5)


def test_restart_cuts_nan_and_infinity():
    """Nothing of a document that overflowed reaches the next one, forward or back."""
    parts, p, s = make(300, 1, 70, torch.float32, packed=False)
    reset = torch.zeros((300, 1), dtype=torch.uint8, device=DEV)
    reset[100] = reset[200] = 1
    parts[2][50, 0, 3] = float("nan")
    parts[2][60, 0, 9] = float("inf")
    s["gh"][150, 0, 11] = float("nan")
    ck = lrs.glr_checkpoints(parts[0])
    h = lrs.glr_fwd(*parts, **p, reset=reset, h0=s["h0"], checkpoints=ck)
    gz = lrs.glr_bwd(*parts, **p, checkpoints=ck, grad_h=s["gh"], reset=reset)
    assert torch.isnan(h[50:100, 0, 3]).all() and torch.isinf(h[60:100, 0, 9]).all()
    assert torch.isfinite(h[100:]).all()
    for t in gz[:3]:
        assert torch.isfinite(t[200:]).all()
        assert torch.isfinite(t[:100, 0, 11]).all()  # gradient of another document's NaN
    assert torch.isnan(gz[2][100:151, 0, 11]).all()
    assert (gz[0][100] == 0).all()
    clean = parts[2].clone()
    clean[:100] = 0
    same = lrs.glr_fwd(parts[0], parts[1], clean, **p, reset=reset, h0=s["h0"])
    np.testing.assert_allclose(f64(same[100:]), f64(h[100:]), rtol=0, atol=0)


def test_every_step_restarts():
    parts, p, s = make(70, 2, 64, torch.float32)
    s["reset"] = torch.ones((70, 2), dtype=torch.uint8, device=DEV)
    h, _, gz = check(parts, p, s)
    assert (gz[0] == 0).all() and (gz[6] == 0).all()


def test_closed_and_open_gates():
    """Gates at both ends: a closed gate gives a = 1 and m = 0 to the last bit,
    whose gradient has to be 0 and not 0/0."""
    parts, p, s = make(90, 2, 34, torch.float32, packed=False)
    parts[0][::3] = -200.0
    parts[0][1::3] = 200.0
    parts[1][::2] = -200.0
    check(parts, p, s)


def test_long_memory():
    """a = 1 - 1e-6: sqrt(1 - a^2) must not lose its digits."""
    parts, p, s = make(256, 1, 64, torch.float32)
    p["decay"] = torch.full_like(p["decay"], float(np.log(np.expm1(1.25e-7))))
    ref = reference(parts, p, s, grad=False)
    h = lrs.glr_fwd(*parts, **p, h0=None)
    b = R.glr(*(f64(t) for t in parts), f64(p["bias_r"]), f64(p["bias_i"]), f64(p["decay"]), 8.0)
    # relative to the inputs' own size (1e-3): 1 - a^2 by subtraction would be 6% off
    assert np.abs(f64(h) - b["h"]).max() <= 1e-5 * np.abs(b["h"]).max()
    close("h", lrs.glr_fwd(*parts, **p, h0=s["h0"]), ref["h"], 1e-5)


def test_empty():
    parts, p, s = make(0, 2, 8, torch.float32, packed=False)
    ck = lrs.glr_checkpoints(parts[0])
    assert ck.shape == (0, 2, 8)
    h, hl = lrs.glr_fwd(*parts, **p, h0=s["h0"], want_h_last=True, checkpoints=ck)
    assert h.shape == (0, 2, 8) and torch.equal(hl, s["h0"])
    gz = lrs.glr_bwd(*parts, **p, checkpoints=ck, grad_h=s["gh"], grad_h_last=s["gl"])
    assert torch.equal(gz[6], s["gl"]) and all((t == 0).all() for t in gz[3:6])


def test_repeatable():
    parts, p, s = make(2000, 1, 200, torch.bfloat16, restart=0.01)
    runs = []
    for _ in range(3):
        ck = lrs.glr_checkpoints(parts[0])
        h = lrs.glr_fwd(*parts, **p, reset=s["reset"], checkpoints=ck)
        runs.append((h, ck, *lrs.glr_bwd(*parts, **p, checkpoints=ck, grad_h=s["gh"],
                                         reset=s["reset"])))
    assert all(torch.equal(u, v) for r in runs[1:] for u, v in zip(runs[0], r))


def test_other_stream():
    parts, p, s = make(500, 2, 128, torch.float32)
    want = lrs.glr_fwd(*parts, **p, h0=s["h0"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = lrs.glr_fwd(*parts, **p, h0=s["h0"])
    st.synchronize()
    assert torch.equal(want, got)


# ---- single tokens -----------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,D", [(1, 1), (3, 37), (64, 1024), (5, 130)])
def test_step(B, D, dtype):
    parts, p, s = make(1, B, D, dtype, seed=B)
    z = [t[0] for t in parts]
    pool = torch.randn(2 * B + 1, D, device=DEV)
    slots = torch.randperm(2 * B + 1, device=DEV)[:B].to(torch.int32)
    if B > 2:
        slots[1], slots[2] = -1, 2 * B + 1  # idle: below and past the pool
    old = pool.clone()
    h = lrs.glr_step(*z, **p, state=pool, slots=slots)
    torch.cuda.synchronize()
    live = [b for b in range(B) if 0 <= int(slots[b]) < 2 * B + 1]
    sl = slots.long()[live]
    ref = R.glr(*(f64(t[live])[None] for t in z), f64(p["bias_r"]), f64(p["bias_i"]),
                f64(p["decay"]), 8.0, None, f64(old[sl]))
    close("state", pool[sl], ref["h_last"], 1e-5)
    close("h", h[live], ref["h"][0], TOL[dtype])
    idle = [b for b in range(B) if b not in live]
    assert (h[idle] == 0).all()
    rest = torch.ones(2 * B + 1, dtype=torch.bool, device=DEV)
    rest[sl] = False
    assert torch.equal(pool[rest], old[rest])


def test_steps_continue_a_prompt():
    """A prompt by glr_fwd, then tokens by glr_step: the states of one long call."""
    parts, p, s = make(80, 4, 64, torch.float32)
    whole, last = lrs.glr_fwd(*parts, **p, want_h_last=True)
    h, state = lrs.glr_fwd(*(t[:70].contiguous() for t in parts), **p, want_h_last=True)
    for t in range(70, 80):
        h = lrs.glr_step(*(v[t] for v in parts), **p, state=state)
        np.testing.assert_allclose(f64(h), f64(whole[t]), rtol=1e-5, atol=1e-6)
    np.testing.assert_allclose(f64(state), f64(last), rtol=1e-5, atol=1e-6)


# ---- refusals ------------------------------------------------------------------

def test_refusals():
    parts, p, s = make(8, 2, 16, torch.float32)
    with pytest.raises(TypeError):
        lrs.glr_fwd(parts[0], parts[1].to(torch.bfloat16), parts[2], **p)
    with pytest.raises(TypeError):
        lrs.glr_fwd(*(t.half() for t in parts), **p)
    with pytest.raises(ValueError):
        lrs.glr_fwd(parts[0], parts[1].contiguous(), parts[2], **p)  # pitches differ
    with pytest.raises(ValueError):
        lrs.glr_fwd(*(t.transpose(1, 2) for t in parts), **p)
    with pytest.raises(ValueError):
        lrs.glr_fwd(*parts, p["bias_r"][:8].contiguous(), p["bias_i"], p["decay"])
    with pytest.raises(ValueError):
        lrs.glr_fwd(*parts, **p, reset=torch.zeros((2, 8), dtype=torch.uint8, device=DEV))
    with pytest.raises(lrs.LrsError):
        lrs.glr_fwd(*parts, **p, c=-1.0)
    with pytest.raises(lrs.LrsError):  # output on top of an input
        cont = [t.contiguous() for t in parts]
        lrs.glr_fwd(*cont, **p, out=cont[2])
    with pytest.raises(TypeError):
        lrs.glr_bwd(*parts, **p, checkpoints=None, grad_h=s["gh"])
    with pytest.raises(lrs.LrsError):  # gradients on top of each other
        ck = lrs.glr_checkpoints(parts[0])
        one = torch.empty((8, 2, 16), device=DEV)
        lrs.glr_bwd(*parts, **p, checkpoints=ck, grad_h=s["gh"], grad_z=(one, one, torch.empty_like(one)))
    with pytest.raises(ValueError):
        lrs.glr_step(*(t[0] for t in parts), **p, state=torch.zeros(1, 16, device=DEV))
