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
