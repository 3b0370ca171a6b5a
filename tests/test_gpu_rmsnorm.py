"""RMS norm with the residual added in, and its 8-bit output, on the GPU against the
plain fp64 form.  Bounds: fp32 results 1e-5 of 1 + |value| (a sum of squares, all of one
sign, over a row and tens of roundings of 6e-8); bf16 results half a unit in the last
place more, 2^-8; the weight's gradient 1e-5 of the sum of its absolute terms (fp32
partial sums of at most 256 rows, joined in fp64).  8 bits: y is known to 1e-6 of itself
(the row's sum of squares to 5e-7 at these widths, and three roundings), so a byte is the
nearest of the grid, or the next one where y / scale is within 2e-6 of a border."""
import math

import pytest
import torch

import linear_recurrence_scan_diagonal_amd as lrs
import block_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = {torch.float32: 1e-5, torch.bfloat16: 2.0 ** -8 + 1e-5}
FP8 = torch.float8_e4m3fn


def f64(t):
    return t.detach().cpu().double()


def close(name, got, ref, tol, scale=None):
    off = (f64(got) - ref).abs() / (1.0 + (ref.abs() if scale is None else scale))
    assert off.max() <= tol, (name, float(off.max()))


def make(rows, D, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = dict(x=(n(rows, D) * (0.2 + 3 * torch.rand(rows, 1, generator=g))).to(dtype), residual=n(rows, D).to(dtype),
             gamma=1 + 0.2 * n(D), gy=n(rows, D).to(dtype), gsum=n(rows, D).to(dtype))
    return {k: v.to(DEV) for k, v in t.items()}


SIZES = [(1, 1), (1, 2), (3, 7), (5, 64), (2, 255), (9, 256), (130, 512), (4, 513), (1, 1023), (67, 1024),
         (5, 1025), (33, 2047), (3, 2048), (7, 2049), (6, 4096), (3, 4099), (2, 8192), (2, 8195),
         (3, 16384), (2, 33000), (5000, 96)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,D", SIZES)
@pytest.mark.parametrize("residual", [False, True])
def test_parity(rows, D, dtype, residual):
    t = make(rows, D, dtype, seed=rows + D)
    res = t["residual"] if residual else None
    y, s, rstd = lrs.rmsnorm_fwd(t["x"], t["gamma"], residual=res, save=True)
    if residual:
        assert torch.equal(s, (t["x"].float() + res.float()).to(dtype))  # one rounding
    else:
        assert s is None
        s = t["x"]
    gsum = t["gsum"] if residual else None
    gx, gg = lrs.rmsnorm_bwd(s, t["gamma"], rstd, t["gy"], grad_sum=gsum)
    torch.cuda.synchronize()
    ref = R.rmsnorm(f64(s), f64(t["gamma"]), 1e-6, f64(t["gy"]), None if gsum is None else f64(gsum))
    close("y", y, ref["y"], TOL[dtype])
    close("rstd", rstd, ref["rstd"], 1e-5)
    close("grad_x", gx, ref["grad_x"], TOL[dtype])
    close("grad_gamma", gg, ref["grad_gamma"], 1e-5, ref["scale_grad_gamma"])


def check_bytes(q, scales, y, group):
    """q and scales against y in fp64."""
    rows, D = y.shape
    step = D if group == 0 else group
    assert scales.shape == (rows, -(-D // step)) and q.dtype == FP8 and q.shape == y.shape
    grid = R.e4m3_grid()
    borders = (grid[1:] + grid[:-1]) / 2
    q, scales = f64(q.float()), f64(scales)
    for i in range(scales.shape[1]):
        part = y[:, i * step:(i + 1) * step]
        top = part.abs().amax(1)
        want = torch.where(top == 0, 1.0, (top / 448).clamp(min=2.0 ** -120))
        assert ((scales[:, i] - want).abs() <= 2e-6 * want).all()
        r = (part / want[:, None]).abs().clamp(max=448.0)
        low, high = (torch.bucketize(r * f, borders) for f in (1 - 2e-6, 1 + 2e-6))
        have = torch.searchsorted(grid, q[:, i * step:(i + 1) * step].abs())
        assert (grid[have.clamp(max=len(grid) - 1)] == q[:, i * step:(i + 1) * step].abs()).all()
        assert ((have >= low) & (have <= high)).all()
        signs = (q[:, i * step:(i + 1) * step] * part) >= 0
        assert signs.all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,D", SIZES)
@pytest.mark.parametrize("group", [0, 128])
def test_8_bits(rows, D, dtype, group):
    t = make(rows, D, dtype, seed=rows + D)
    residual = t["residual"] if (rows + D) % 2 else None
    q, scales, s = lrs.rmsnorm_fwd_fp8(t["x"], t["gamma"], residual=residual, group=group)
    y, s2, _ = lrs.rmsnorm_fwd(t["x"], t["gamma"], residual=residual)
    if residual is None:
        assert s is None
        s = t["x"]
    else:
        assert torch.equal(s, s2)
    check_bytes(q, scales, R.rmsnorm(f64(s), f64(t["gamma"]), 1e-6)["y"], group)


@pytest.mark.parametrize("group", [0, 128])
def test_8_bits_of_nothing_and_of_small_values(group):
    """Groups of zeros have scale 1 and bytes 0; values too small for a normal inverse keep a
    finite one."""
    t = make(4, 300, torch.float32)
    t["gamma"][:128] = 0.0
    t["x"][1] = 0.0
    q, scales, _ = lrs.rmsnorm_fwd_fp8(t["x"], t["gamma"], group=group)
    check_bytes(q, scales, R.rmsnorm(f64(t["x"]), f64(t["gamma"]), 1e-6)["y"], group)
    assert (scales[1] == 1.0).all() and (q[1].float() == 0).all()
    tiny = torch.full_like(t["gamma"], 1e-38)
    q, scales, _ = lrs.rmsnorm_fwd_fp8(t["x"], tiny, group=group)
    assert (scales[[0, 2, 3]] == 2.0 ** -120).all() and torch.isfinite(q.float()).all()


@pytest.mark.parametrize("D", [200, 3000, 40000])
def test_not_finite_stays_in_its_row(D):
    t = make(5, D, torch.float32, seed=D)
    t["x"][1, 7] = math.nan
    t["x"][3, 150] = math.inf
    y, _, rstd = lrs.rmsnorm_fwd(t["x"], t["gamma"], save=True)
    gx, _ = lrs.rmsnorm_bwd(t["x"], t["gamma"], rstd, t["gy"])
    keep = [0, 2, 4]
    assert torch.isnan(y[1]).all() and torch.isnan(gx[1]).all() and torch.isnan(y[3, 150])
    assert torch.isfinite(y[keep]).all() and torch.isfinite(gx[keep]).all()
    for group in (0, 128):
        q, scales, _ = lrs.rmsnorm_fwd_fp8(t["x"], t["gamma"], group=group)
        assert torch.isfinite(scales[keep]).all() and torch.isfinite(q[keep].float()).all()
        assert torch.isnan(scales[1]).all() and torch.isnan(q[1].float()).all()
        part = slice(128, min(D, 256)) if group else slice(0, D)
        assert torch.isnan(q[3, part].float()).all()
        assert not torch.isfinite(scales[3, 1 if group else 0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [100, 1024, 2051, 20000])
def test_in_place(D, dtype):
    """The residual stream in place, and gradients over their inputs: same bits."""
    t = make(6, D, dtype, seed=D)
    y, s, rstd = lrs.rmsnorm_fwd(t["x"], t["gamma"], residual=t["residual"], save=True)
    q, sc, _ = lrs.rmsnorm_fwd_fp8(t["x"], t["gamma"], residual=t["residual"])
    for which in ("x", "residual"):
        u = {k: v.clone() for k, v in t.items()}
        y2, s2, _ = lrs.rmsnorm_fwd(u["x"], u["gamma"], residual=u["residual"], out_sum=u[which])
        assert s2 is u[which] and torch.equal(s2, s) and torch.equal(y2, y)
        u = {k: v.clone() for k, v in t.items()}
        q2, sc2, s2 = lrs.rmsnorm_fwd_fp8(u["x"], u["gamma"], residual=u["residual"], out_sum=u[which])
        assert torch.equal(s2, s) and torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(sc2, sc)
    gx, gg = lrs.rmsnorm_bwd(s, t["gamma"], rstd, t["gy"], grad_sum=t["gsum"])
    for which in ("gy", "gsum"):
        u = {k: v.clone() for k, v in t.items()}
        g2 = lrs.rmsnorm_bwd(s, u["gamma"], rstd, u["gy"], grad_sum=u["gsum"], out=u[which])
        assert torch.equal(g2[0], gx) and torch.equal(g2[1], gg)


def test_misaligned_views():
    t = make(5, 200, torch.bfloat16)
    buf = torch.empty(5 * 200 + 1, dtype=torch.bfloat16, device=DEV)
    x1 = buf[1:].view(5, 200)
    x1.copy_(t["x"])
    assert torch.equal(lrs.rmsnorm_fwd(t["x"], t["gamma"])[0], lrs.rmsnorm_fwd(x1, t["gamma"])[0])
    out = torch.empty(5 * 200 + 1, dtype=torch.uint8, device=DEV)[1:].view(FP8).view(5, 200)
    a, b = lrs.rmsnorm_fwd_fp8(t["x"], t["gamma"]), lrs.rmsnorm_fwd_fp8(x1, t["gamma"], out=out)
    assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])


def test_more_axes_and_empty():
    t = make(12, 64, torch.float32)
    y = lrs.rmsnorm_fwd(t["x"].view(3, 4, 64), t["gamma"])[0]
    assert torch.equal(y.view(12, 64), lrs.rmsnorm_fwd(t["x"], t["gamma"])[0])
    e = torch.empty((0, 64), device=DEV)
    y, s, rstd = lrs.rmsnorm_fwd(e, t["gamma"], save=True)
    gx, gg = lrs.rmsnorm_bwd(e, t["gamma"], rstd, e)
    assert y.shape == (0, 64) and (gg == 0).all()
    assert lrs.rmsnorm_fwd_fp8(e, t["gamma"])[1].shape == (0, 1)


def test_gradient_against_differences():
    """Central differences of the fp64 form at the point, along one direction."""
    t = make(7, 130, torch.float32, seed=3)
    _, _, rstd = lrs.rmsnorm_fwd(t["x"], t["gamma"], save=True)
    gx, gg = lrs.rmsnorm_bwd(t["x"], t["gamma"], rstd, t["gy"])
    g = torch.Generator().manual_seed(1)
    dx, dg = torch.randn(7, 130, generator=g).double(), torch.randn(130, generator=g).double()
    f = lambda h: (R.rmsnorm(f64(t["x"]) + h * dx, f64(t["gamma"]) + h * dg, 1e-6)["y"] * f64(t["gy"])).sum()  # noqa: E731
    slope = (f(1e-5) - f(-1e-5)) / 2e-5
    terms = (f64(gx) * dx).abs().sum() + (f64(gg) * dg).abs().sum()
    assert abs((f64(gx) * dx).sum() + (f64(gg) * dg).sum() - slope) <= 1e-5 * terms


def test_repeatable():
    t = make(3000, 384, torch.bfloat16)
    _, _, rstd = lrs.rmsnorm_fwd(t["x"], t["gamma"], save=True)
    runs = [lrs.rmsnorm_bwd(t["x"], t["gamma"], rstd, t["gy"]) for _ in range(3)]
    assert all(torch.equal(u, v) for r in runs[1:] for u, v in zip(runs[0], r))


def test_refusals():
    t = make(4, 32, torch.float32)
    with pytest.raises(TypeError):
        lrs.rmsnorm_fwd(t["x"].half(), t["gamma"])
    with pytest.raises(TypeError):
        lrs.rmsnorm_fwd(t["x"], t["gamma"].to(torch.bfloat16))
    with pytest.raises(TypeError):
        lrs.rmsnorm_fwd(t["x"], None)
    with pytest.raises(ValueError):
        lrs.rmsnorm_fwd(t["x"].t(), t["gamma"])
    with pytest.raises(ValueError):
        lrs.rmsnorm_fwd(t["x"], t["gamma"][:16].contiguous())
    with pytest.raises(lrs.LrsError):
        lrs.rmsnorm_fwd(t["x"], t["gamma"], eps=-1.0)
    with pytest.raises(lrs.LrsError):
        lrs.rmsnorm_fwd(t["x"], t["gamma"], out=t["x"])
    with pytest.raises(ValueError):
        lrs.rmsnorm_fwd_fp8(t["x"], t["gamma"], group=64)
    with pytest.raises(TypeError):
        lrs.rmsnorm_fwd_fp8(t["x"], t["gamma"], out=torch.empty(4, 32, dtype=torch.uint8, device=DEV))
    with pytest.raises(lrs.LrsError):  # grad_x over s
        lrs.rmsnorm_bwd(t["x"], t["gamma"], torch.ones(4, device=DEV), t["gy"], out=t["x"])
    with pytest.raises(TypeError):
        lrs.rmsnorm_bwd(t["x"], t["gamma"], None, t["gy"])
