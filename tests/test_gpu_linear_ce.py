"""Cross entropy of a linear head on the GPU against the plain fp64 form.

Bounds.  The logits are fp32 sums of exact products: with K terms of size s the
rounding is at most K 2^-24 of their absolute sum, far below 1e-5 of 1 + |value|
for loss and lse at these sizes.  The gradients are sums of G_k times an operand;
in bf16, G is rounded to 2^-8 of itself at most, the result to 2^-8 of itself:
2^-8 of the sum of the absolute terms, plus 2^-8 of the value.  In fp32 the
absolute error of a logit, 1e-6 of its absolute sum (at most 20 here), becomes a
relative one of G: 3e-5 of the sum of absolute terms."""
import numpy as np
import pytest
import torch

import linear_recurrence_scan_diagonal_amd as lrs
import lm_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def make(N, V, D, dtype, seed=0, ignored=0.2, uniform=True):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, w = n(N, D).to(dtype), (n(V, D) * 2 / D ** 0.5).to(dtype)
    target = torch.randint(0, V, (N,), generator=g)
    target[torch.rand(N, generator=g) < ignored] = -100
    gl = torch.full((N,), 1.0 / max(1, N)) if uniform else n(N)
    return [t.to(DEV) for t in (x, w, target, gl)]


def check_forward(x, w, target, loss, lse, ref):
    for name, t in (("loss", loss), ("lse", lse)):
        off = np.abs(f64(t) - ref[name]) / (1 + np.abs(ref[name]))
        assert off.max() <= 1e-5, (name, off.max())


def check_grads(dtype, gx, gw, ref):
    tol = 2.0 ** -8 if dtype == torch.bfloat16 else 3e-5
    for name, t in (("grad_x", gx), ("grad_w", gw)):
        r, s = ref[name], ref["scale_" + name]
        off = np.abs(f64(t) - r) - tol * (s + np.abs(r))
        assert np.isfinite(f64(t)).all() and off.max() <= 1e-30, (name, off.max())


def check(x, w, target, gl):
    loss, lse = lrs.linear_ce_fwd(x, w, target)
    gx, gw = lrs.linear_ce_bwd(x, w, target, lse, gl)
    both = lrs.linear_ce_fwd_bwd(x, w, target, gl)
    torch.cuda.synchronize()
    ref = R.linear_ce(f64(x), f64(w), target.cpu().numpy(), f64(gl))
    check_forward(x, w, target, loss, lse, ref)
    check_grads(x.dtype, gx, gw, ref)
    check_forward(x, w, target, both[0], both[1], ref)
    check_grads(x.dtype, both[2], both[3], ref)
    ign = (target < 0) | (target >= w.shape[0])
    assert (loss[ign] == 0).all() and (gx[ign] == 0).all() and (both[2][ign] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,V,D", [
    (1, 1, 1), (1, 5, 3), (2, 130, 64), (7, 1000, 33), (64, 128, 32), (65, 129, 65), (100, 257, 96),
    (129, 2000, 128), (33, 4097, 100), (300, 777, 200), (512, 512, 512)])
def test_parity(N, V, D, dtype):
    check(*make(N, V, D, dtype, seed=N + V))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_tiles(dtype):
    """Shapes whose logits and gradients take the large tiles."""
    check(*make(2050, 8200, 136, dtype, seed=3))
    check(*make(700, 12000, 1060, dtype, seed=4))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_weights_per_row(dtype):
    """grad_loss of any sign and size a row, zero among them."""
    x, w, target, gl = make(200, 600, 72, dtype, uniform=False)
    gl[::7] = 0.0
    gl[3] = 50.0
    check(x, w, target, gl)


def test_nothing_counts():
    x, w, target, gl = make(70, 300, 40, torch.bfloat16)
    target[:] = -1
    target[::2] = 300  # past the last class
    loss, lse, gx, gw = lrs.linear_ce_fwd_bwd(x, w, target, gl)
    assert (loss == 0).all() and (gx == 0).all() and (gw == 0).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ignored_rows_may_hold_anything(dtype):
    """NaN and infinities in ignored rows (and in their grad_loss) reach no gradient."""
    x, w, target, gl = make(150, 500, 64, dtype, ignored=0.4)
    clean = lrs.linear_ce_fwd_bwd(x, w, target, gl)
    ign = target < 0
    x2, gl2 = x.clone(), gl.clone()
    x2[ign] = float("nan")
    x2[torch.nonzero(ign)[0, 0]] = float("inf")
    gl2[ign] = float("nan")
    got = lrs.linear_ce_fwd_bwd(x2, w, target, gl2)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2]) and torch.equal(got[3], clean[3])


def test_extreme_logits():
    """One class far above all: the sum must not overflow, p is 1 or 0."""
    x, w, target, gl = make(40, 300, 32, torch.float32, ignored=0.0)
    w[17] = w[17] * 400.0
    loss, lse, gx, gw = lrs.linear_ce_fwd_bwd(x, w, target, gl)
    ref = R.linear_ce(f64(x), f64(w), target.cpu().numpy(), f64(gl))
    off = np.abs(f64(lse) - ref["lse"]) / (1 + np.abs(ref["lse"]))
    assert off.max() <= 1e-5 and torch.isfinite(gx).all() and torch.isfinite(gw).all()


def test_pieces_of_the_vocabulary():
    """Enough rows and classes that G is made in several pieces."""
    N, V, D = 16384, 33000, 64
    g = torch.Generator(device=DEV).manual_seed(0)
    x = torch.randn(N, D, generator=g, device=DEV).to(torch.bfloat16)
    w = (torch.randn(V, D, generator=g, device=DEV) / 4).to(torch.bfloat16)
    target = torch.randint(0, V, (N,), generator=g, device=DEV)
    target[::9] = -100
    gl = torch.full((N,), 1.0 / N, device=DEV)
    loss, lse, gx, gw = lrs.linear_ce_fwd_bwd(x, w, target, gl)
    x64, w64 = x.double(), w.double()
    want_lse = torch.logsumexp(x64 @ w64.t(), 1)
    assert ((lse.double() - want_lse).abs() / (1 + want_lse.abs())).max() <= 1e-5
    p = torch.exp(x64 @ w64.t() - want_lse[:, None])
    counts = target >= 0
    rows = torch.nonzero(counts)[:, 0]
    p[rows, target[rows]] -= 1.0
    p *= (gl.double() * counts)[:, None]
    for got, a, b in ((gx, p, w64), (gw, p.t().contiguous(), x64)):
        want, scale = a @ b, a.abs() @ b.abs()
        assert ((got.double() - want).abs() - 2.0 ** -8 * (scale + want.abs())).max() <= 1e-30


def test_misaligned_views():
    x, w, target, gl = make(60, 200, 64, torch.bfloat16)
    bx, bw = (torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV) for t in (x, w))
    x1, w1 = bx[1:].view_as(x), bw[1:].view_as(w)
    x1.copy_(x)
    w1.copy_(w)
    a, b = lrs.linear_ce_fwd_bwd(x, w, target, gl), lrs.linear_ce_fwd_bwd(x1, w1, target, gl)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_no_rows():
    x, w, target, gl = make(0, 30, 16, torch.bfloat16)
    loss, lse, gx, gw = lrs.linear_ce_fwd_bwd(x, w, target, gl)
    assert loss.shape == (0,) and (gw == 0).all()


def test_repeatable():
    args = make(900, 5000, 192, torch.bfloat16)
    runs = [lrs.linear_ce_fwd_bwd(*args) for _ in range(3)]
    assert all(torch.equal(u, v) for r in runs[1:] for u, v in zip(runs[0], r))


def test_other_stream_and_given_workspace():
    args = make(200, 1000, 64, torch.bfloat16)
    want = lrs.linear_ce_fwd_bwd(*args)
    nbytes = lrs.load().lrs_linear_ce_workspace_bytes(200, 1000, 64, 1, 1)
    ws = torch.full((nbytes,), 255, dtype=torch.uint8, device=DEV)  # whatever was there before
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = lrs.linear_ce_fwd_bwd(*args, workspace=ws)
    st.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, got))


def test_refusals():
    x, w, target, gl = make(8, 20, 16, torch.bfloat16)
    with pytest.raises(TypeError):
        lrs.linear_ce_fwd(x.half(), w.half(), target)
    with pytest.raises(TypeError):
        lrs.linear_ce_fwd(x, w, target.int())
    with pytest.raises(ValueError):
        lrs.linear_ce_fwd(x, w[:, :8].contiguous(), target)
    with pytest.raises(ValueError):
        lrs.linear_ce_fwd(x, w, target[:4].contiguous())
    with pytest.raises(lrs.LrsError):
        lrs.linear_ce_fwd(x, w[:0].contiguous(), target)
    with pytest.raises(lrs.LrsError):
        lrs.linear_ce_fwd_bwd(x, w, target, gl, out=(x, torch.empty_like(w)))
