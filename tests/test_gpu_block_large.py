"""The kernels that calls of many rows take, against the plain fp64 form: log probabilities of
wide rows by 256 threads a row (from twice as many rows as compute units on), and the RMS norm
with nontemporal accesses (from 512 MiB on) with a residual and its gradient.

Bounds: those of test_gpu_logprobs and test_gpu_rmsnorm.  Rows do not depend on each other, so
the references are of some rows; the weight's gradient is of all, in fp64 on the device."""
import pytest
import torch

import linear_recurrence_scan_diagonal_amd as lrs
import block_ref as R
import test_gpu_logprobs as L
import test_gpu_rmsnorm as N

pytestmark = pytest.mark.gpu
DEV = "cuda"


def some(n):
    return sorted({0, 1, 2, 3, n // 3, n // 2, n - 2, n - 1, *range(5, n, max(1, n // 40))})


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,top", [(8191, 0), (8193, 5), (20011, 20), (33333, 64), (50000, 1)])
@pytest.mark.parametrize("how", ["random", "ties", "masked", "rising"])
def test_wide_rows(V, top, how, dtype):
    rows = 700
    g = torch.Generator(device=DEV).manual_seed(V)
    x = 3 * torch.randn(rows, V, generator=g, device=DEV)
    if how == "ties":
        x = x.round()
    elif how == "rising":  # every group of a thread has a larger value than the one before
        x = x * 0.01 + torch.arange(V, device=DEV) * (20.0 / V)
    x = x.to(dtype)
    target = torch.randint(0, V, (rows,), generator=g, device=DEV)
    target[::7] = -100
    if how == "masked":
        x[:, 1::3] = -torch.inf
        x[5::50, 64:] = -torch.inf  # hardly any token left
        target[target % 3 == 1] -= 1
        target[5::50] = 0
    gl, ge = (torch.randn(rows, generator=g, device=DEV) for _ in range(2))
    logprob, entropy, lse, ids, tops = lrs.logprobs_fwd(x, target, top=top)
    grad = lrs.logprobs_bwd(x, target, lse, entropy, gl, ge)
    at = torch.tensor(sorted({*some(rows), 55, 105, 655}), device=DEV)
    f = lambda t: t[at].cpu().double()  # noqa: E731
    ref = R.logprobs(f(x), target[at].cpu(), f(gl), f(ge))
    for name, got in (("logprob", logprob), ("entropy", entropy), ("lse", lse)):
        L.close(name, got[at], ref[name], 2e-6)
    if top:
        want = R.tops(f(x), top)
        assert torch.equal(ids[at].cpu(), want)
        L.close("tops", tops[at], ref["lp"].gather(1, want), 2e-6)
    lp = ref["lp"].clamp(min=-200)
    terms = torch.exp(ref["lp"]) * (f(gl).abs()[:, None] + f(ge).abs()[:, None] * (lp.abs() + ref["entropy"][:, None]))
    want = ref["grad_logits"]
    bound = 8e-6 * (terms + want.abs()) + 1e-38 + (2.0 ** -8 * want.abs() if dtype == torch.bfloat16 else 0)
    assert ((f(grad) - want).abs() <= bound).all()


# threads a row and 16-byte groups a thread: 64 x 2, 64 x 4, 256 x 2, 256 x 4, 1024 x 2 (forward; by passes backward)
@pytest.mark.parametrize("dtype,rows,D", [(torch.bfloat16, 90001, 1000), (torch.bfloat16, 50021, 1903), (torch.bfloat16, 24007, 4096),
                                          (torch.bfloat16, 12007, 8100), (torch.bfloat16, 6007, 16200), (torch.float32, 90001, 505),
                                          (torch.float32, 45001, 1023), (torch.float32, 23003, 2047), (torch.float32, 12007, 4091),
                                          (torch.float32, 6007, 8100)])
def test_large_norm(rows, D, dtype):
    assert rows * D * 3 * (torch.finfo(dtype).bits // 8) >= 512 << 20
    g = torch.Generator(device=DEV).manual_seed(D)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, residual, gy, gsum = (n(rows, D).to(dtype) for _ in range(4))
    gamma = 1 + 0.2 * n(D)
    y, s, rstd = lrs.rmsnorm_fwd(x, gamma, residual=residual, save=True)
    q, scales, s8 = lrs.rmsnorm_fwd_fp8(x, gamma, residual=residual)
    assert torch.equal(s8, s) and torch.equal(s, (x.float() + residual.float()).to(dtype))
    gx, gg = lrs.rmsnorm_bwd(s, gamma, rstd, gy, grad_sum=gsum)
    at = torch.tensor(some(rows), device=DEV)
    f = lambda t: t[at].cpu().double()  # noqa: E731
    ref = R.rmsnorm(f(s), gamma.cpu().double(), 1e-6, f(gy), f(gsum))
    N.close("y", y[at], ref["y"], N.TOL[dtype])
    N.close("rstd", rstd[at], ref["rstd"], 1e-5)
    N.close("grad_x", gx[at], ref["grad_x"], N.TOL[dtype])
    N.check_bytes(q.view(torch.uint8)[at].view(torch.float8_e4m3fn), scales[at], ref["y"], 128)
    want, size = torch.zeros(D, dtype=torch.float64, device=DEV), torch.zeros(D, dtype=torch.float64, device=DEV)
    for a in range(0, rows, 4096):
        v = s[a:a + 4096].double()
        t = gy[a:a + 4096].double() * v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6)
        want += t.sum(0)
        size += t.abs().sum(0)
    N.close("grad_gamma", gg, want.cpu(), 1e-5, size.cpu())
    # in place, and the same rows in a call of their own
    y1, s1, rstd1 = lrs.rmsnorm_fwd(x, gamma, residual=residual, save=True, out_sum=x)
    assert s1 is x and torch.equal(s1, s) and torch.equal(y1, y) and torch.equal(rstd1, rstd)
    gx1, gg1 = lrs.rmsnorm_bwd(s, gamma, rstd, gy, grad_sum=gsum, out=gsum)
    assert torch.equal(gx1, gx) and torch.equal(gg1, gg)
