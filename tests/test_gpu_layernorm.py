"""Layer norm with the residual added in, on the GPU, against the plain fp64
form.  Bounds: fp32 results 1e-5 of 1 + |value| (sums over a row and tens of
roundings of 6e-8 of the normalised values); bf16 results half a unit in the
last place more, 2^-8; the weight's gradients 1e-5 of the sum of their absolute
terms (fp32 partial sums of at most some hundred rows, joined in fp64)."""
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


def close(name, got, ref, tol, scale=None):
    off = np.abs(f64(got) - ref) / (1.0 + (np.abs(ref) if scale is None else scale))
    assert off.max() <= tol, (name, off.max())


def make(R_, D, dtype, seed=0, mean=1.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = dict(x=(n(R_, D) + mean * n(R_, 1)).to(dtype), residual=n(R_, D).to(dtype),
             gamma=1 + 0.2 * n(D), beta=0.2 * n(D), gy=n(R_, D).to(dtype), gsum=n(R_, D).to(dtype))
    return {k: v.to(DEV) for k, v in t.items()}


def check(t, residual, beta=True, eps=1e-5):
    dtype = t["x"].dtype
    res = t["residual"] if residual else None
    be = t["beta"] if beta else None
    y, s, mean, rstd = lrs.layernorm_fwd(t["x"], t["gamma"], be, residual=res, eps=eps, save=True)
    assert (s is None) == (res is None)
    if residual:
        want = (t["x"].float() + res.float()).to(dtype)  # one rounding
        assert torch.equal(s, want)
    s = t["x"] if s is None else s
    gsum = t["gsum"] if residual else None
    gx, gg, gb = lrs.layernorm_bwd(s, t["gamma"], mean, rstd, t["gy"], grad_sum=gsum,
                                   want_grad_beta=beta)
    torch.cuda.synchronize()
    ref = R.layernorm(f64(s), f64(t["gamma"]), f64(be) if beta else None, eps, f64(t["gy"]),
                      None if gsum is None else f64(gsum))
    close("y", y, ref["y"], TOL[dtype])
    close("mean", mean, ref["mean"], 1e-5)
    close("rstd", rstd, ref["rstd"], 1e-5)
    close("grad_x", gx, ref["grad_x"], TOL[dtype])
    close("grad_gamma", gg, ref["grad_gamma"], 1e-5, ref["scale_grad_gamma"])
    if beta:
        close("grad_beta", gb, ref["grad_beta"], 1e-5, ref["scale_grad_beta"])
    else:
        assert gb is None


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,D", [
    (1, 1), (1, 2), (3, 7), (5, 64), (2, 255), (9, 256), (130, 512), (4, 513), (1, 1023), (67, 1024),
    (5, 1025), (33, 2047), (3, 2048), (7, 2049), (6, 4096), (3, 4099), (2, 8192), (2, 8195),
    (3, 16384), (2, 33000), (5000, 96)])
@pytest.mark.parametrize("residual", [False, True])
def test_parity(rows, D, dtype, residual):
    check(make(rows, D, dtype, seed=rows + D), residual, beta=(rows + D) % 3 != 0)


def test_large_mean():
    """Rows whose mean is a thousand times their spread: the variance is taken
    about the mean (its square would cancel).  The inputs' own grid at 1000 is
    6e-5, and the mean is known to 6e-5 of them."""
    t = make(20, 300, torch.float32, mean=0.0)
    t["x"] = t["x"] + 1000.0
    y, _, mean, rstd = lrs.layernorm_fwd(t["x"], t["gamma"], t["beta"], save=True)
    ref = R.layernorm(f64(t["x"]), f64(t["gamma"]), f64(t["beta"]), 1e-5)
    close("rstd", rstd, ref["rstd"], 1e-5)
    close("y", y, ref["y"], 3 * 6e-5)


def test_constant_rows():
    """No variance: rstd = 1 / sqrt(eps), y = beta."""
    t = make(4, 130, torch.float32)
    t["x"] = torch.full_like(t["x"], 3.0)
    y, _, _, rstd = lrs.layernorm_fwd(t["x"], t["gamma"], t["beta"], save=True)
    assert torch.equal(y, t["beta"].expand(4, 130))
    np.testing.assert_allclose(f64(rstd), 1 / np.sqrt(1e-5), rtol=1e-6)


def test_nan_stays_in_its_row():
    t = make(9, 200, torch.float32)
    t["x"][4, 7] = float("nan")
    y, _, mean, rstd = lrs.layernorm_fwd(t["x"], t["gamma"], t["beta"], save=True)
    gx, _, _ = lrs.layernorm_bwd(t["x"], t["gamma"], mean, rstd, t["gy"])
    keep = [r for r in range(9) if r != 4]
    assert torch.isnan(y[4]).all() and torch.isfinite(y[keep]).all()
    assert torch.isnan(gx[4]).all() and torch.isfinite(gx[keep]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [100, 1024, 2051, 20000])
def test_in_place(D, dtype):
    """The residual stream in place, and gradients over their inputs: same bits."""
    t = make(6, D, dtype, seed=D)
    y, s, mean, rstd = lrs.layernorm_fwd(t["x"], t["gamma"], t["beta"], residual=t["residual"], save=True)
    for which in ("x", "residual"):
        u = {k: v.clone() for k, v in t.items()}
        y2, s2, _, _ = lrs.layernorm_fwd(u["x"], u["gamma"], u["beta"], residual=u["residual"],
                                         out_sum=u[which])
        assert s2 is u[which] and torch.equal(s2, s) and torch.equal(y2, y)
    gx, gg, gb = lrs.layernorm_bwd(s, t["gamma"], mean, rstd, t["gy"], grad_sum=t["gsum"])
    for which in ("gy", "gsum"):
        u = {k: v.clone() for k, v in t.items()}
        g2 = lrs.layernorm_bwd(s, u["gamma"], mean, rstd, u["gy"], grad_sum=u["gsum"], out=u[which])
        assert torch.equal(g2[0], gx) and torch.equal(g2[1], gg) and torch.equal(g2[2], gb)


def test_misaligned_views():
    t = make(5, 200, torch.bfloat16)
    buf = torch.empty(5 * 200 + 1, dtype=torch.bfloat16, device=DEV)
    x1 = buf[1:].view(5, 200)
    x1.copy_(t["x"])
    a = lrs.layernorm_fwd(t["x"], t["gamma"], t["beta"])[0]
    assert torch.equal(a, lrs.layernorm_fwd(x1, t["gamma"], t["beta"])[0])


def test_more_axes_and_empty():
    t = make(12, 64, torch.float32)
    y = lrs.layernorm_fwd(t["x"].view(3, 4, 64), t["gamma"], t["beta"])[0]
    assert torch.equal(y.view(12, 64), lrs.layernorm_fwd(t["x"], t["gamma"], t["beta"])[0])
    e = torch.empty((0, 64), device=DEV)
    y, s, mean, rstd = lrs.layernorm_fwd(e, t["gamma"], t["beta"], save=True)
    assert y.shape == (0, 64)
    gx, gg, gb = lrs.layernorm_bwd(e, t["gamma"], mean, rstd, e)
    assert (gg == 0).all() and (gb == 0).all()


def test_repeatable():
    t = make(3000, 384, torch.bfloat16)
    _, _, mean, rstd = lrs.layernorm_fwd(t["x"], t["gamma"], t["beta"], save=True)
    runs = [lrs.layernorm_bwd(t["x"], t["gamma"], mean, rstd, t["gy"]) for _ in range(3)]
    assert all(torch.equal(u, v) for r in runs[1:] for u, v in zip(runs[0], r))


def test_refusals():
    t = make(4, 32, torch.float32)
    with pytest.raises(TypeError):
        lrs.layernorm_fwd(t["x"].half(), t["gamma"])
    with pytest.raises(TypeError):
        lrs.layernorm_fwd(t["x"], t["gamma"].to(torch.bfloat16))
    with pytest.raises(ValueError):
        lrs.layernorm_fwd(t["x"].t(), t["gamma"])
    with pytest.raises(ValueError):
        lrs.layernorm_fwd(t["x"], t["gamma"][:16].contiguous())
    with pytest.raises(lrs.LrsError):
        lrs.layernorm_fwd(t["x"], t["gamma"], eps=-1.0)
    with pytest.raises(lrs.LrsError):
        lrs.layernorm_fwd(t["x"], t["gamma"], out=t["x"])
    with pytest.raises(lrs.LrsError):  # grad_x over s
        m = torch.zeros(4, device=DEV)
        lrs.layernorm_bwd(t["x"], t["gamma"], m, m + 1, t["gy"], out=t["x"])
