"""Log probabilities of more rows than fit a grid of 1024 threads a row, up to the most that
are supported.  Bounds: those of test_gpu_logprobs, 2e-6 of 1 + |value| (the gradient's 8e-6
of its terms, each of at most 2 here)."""
import pytest
import torch

import linear_recurrence_scan_diagonal_amd as lrs
import block_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("N,V", [((1 << 22) - 1, 3), (1 << 22, 3), ((1 << 22) + 5, 2), ((1 << 24) - 1, 2)])
def test_many_rows(N, V):
    g = torch.Generator().manual_seed(V)
    logits = torch.randn(N, V, generator=g)
    target = torch.randint(-1, V, (N,), generator=g)
    gl = torch.rand(N, generator=g)
    ref = R.logprobs(logits.double(), target, gl.double())
    out = lrs.logprobs_fwd(logits.to(DEV), target.to(DEV), top=1)
    for name, x in zip(("logprob", "entropy", "lse"), out):
        assert ((x.cpu().double() - ref[name]).abs() <= 2e-6 * (1 + ref[name].abs())).all(), name
    assert torch.equal(out[3][:, 0].cpu(), logits.argmax(1))
    grad = lrs.logprobs_bwd(logits.to(DEV), target.to(DEV), out[2], None, gl.to(DEV))
    assert ((grad.cpu().double() - ref["grad_logits"]).abs() <= 1.6e-5).all()


def test_far_from_0_costs_one_more_reading():
    """The gradient sums a row again whose lse is far from 0: that is one more reading of the row,
    half as much again as the call's own reads and writes, whatever the row's width.  Bound: four times
    the call near 0."""
    N, V = 1000, 150000
    x = torch.randn(N, V, device=DEV)
    target = torch.zeros(N, dtype=torch.int64, device=DEV)
    gl, out = torch.ones(N, device=DEV), torch.empty_like(x)
    took = []
    for _ in range(2):
        lse = lrs.logprobs_fwd(x, target)[2]
        runs = []
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            lrs.logprobs_bwd(x, target, lse, None, gl, out=out)
            b.record()
            torch.cuda.synchronize()
            runs.append(a.elapsed_time(b))
        took.append(min(runs))
        x += 1000.0
    assert took[1] <= 4 * took[0], took


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,V", [(1, 40001), (30, 40001), (300, 50021), (1100, 20011)])
def test_far_from_0_in_pieces(N, V, dtype):
    """Rows far from 0, near it and wholly masked together, in every number of pieces: out of
    place as in place, bit for bit."""
    g = torch.Generator(device=DEV).manual_seed(N)
    x = 3 * torch.randn(N, V, generator=g, device=DEV)
    x[::2] += 1000.0
    x[7::9] = -torch.inf
    x = x.to(dtype)
    target = torch.randint(0, V, (N,), generator=g, device=DEV)
    gl, ge = (torch.randn(N, generator=g, device=DEV) for _ in range(2))
    _, entropy, lse, _, _ = lrs.logprobs_fwd(x, target)
    apart = lrs.logprobs_bwd(x, target, lse, entropy, gl, ge)
    lrs.logprobs_bwd(x, target, lse, entropy, gl, ge, out=x)
    kind = torch.int32 if dtype == torch.float32 else torch.int16
    nan = torch.isnan(x)
    assert torch.equal(torch.isnan(apart), nan) and torch.equal(apart.view(kind)[~nan], x.view(kind)[~nan])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [4, 520])
def test_flat_wide_rows(N, dtype):
    """Rows of equal logits below a first few: every addition to a thread's sum rounds the same way.
    A thread of 256 has 879 groups of fp32, whose sum is known to 879 2^-25 = 2.6e-5 of itself, and lse
    to as much: 2e-6 of 1 + |lse|, which is 14."""
    V = 900001
    x = torch.zeros(N, V, dtype=dtype, device=DEV)
    target = torch.zeros(N, dtype=torch.int64, device=DEV)
    for low in (-0.3, -0.7, -1.0, -1.3, -2.1):
        x[:, 8192:] = low
        ref = R.logprobs(x[:1].cpu().double(), target[:1].cpu())
        logprob, entropy, lse, _, _ = lrs.logprobs_fwd(x, target)
        for name, got in (("logprob", logprob), ("entropy", entropy), ("lse", lse)):
            assert (got == got[0]).all()
            off = abs(float(got[0]) - float(ref[name][0])) / (1 + abs(float(ref[name][0])))
            assert off <= 2e-6, (name, low, off)
