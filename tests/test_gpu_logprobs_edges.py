"""Log probabilities where a row's largest logit is far from 0 or the type's lowest value.

Bounds: as for ordinary logits in what is relative to the row's maximum; lse itself is off
by one rounding of its value, 2^-24 |lse|."""
import pytest
import torch

import linear_recurrence_scan_diagonal_amd as lrs
import block_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def f64(t):
    return t.detach().cpu().double()


def run(logits, target, top=0, in_place=False, seed=3):
    N, V = logits.shape
    g = torch.Generator().manual_seed(seed)
    gl, ge = torch.randn(N, generator=g), torch.randn(N, generator=g)
    # in 64 bits too the sum's logarithm would be lost beside a maximum of 1e38
    m = f64(logits).max(1).values
    ref = R.logprobs(f64(logits) - m[:, None], target.cpu(), gl.double(), ge.double())
    ref["lse"] = ref["lse"] + m
    logprob, entropy, lse, ids, tops = lrs.logprobs_fwd(logits, target, top=top)
    for name, got in (("logprob", logprob), ("entropy", entropy)):
        assert ((f64(got) - ref[name]).abs() <= 2e-6 * (1 + ref[name].abs())).all(), name
    assert ((f64(lse) - ref["lse"]).abs() <= 2e-6 * (1 + ref["entropy"].abs()) + 2.0 ** -23 * ref["lse"].abs()).all()
    if top:
        want = R.tops(f64(logits), top)
        assert torch.equal(ids.cpu(), want)
        lp = ref["lp"].gather(1, want)
        assert ((f64(tops) - lp).abs() <= 2e-6 * (1 + lp.abs())).all()
    lp = ref["lp"]
    out = lrs.logprobs_bwd(logits, target, lse, entropy, gl.to(DEV), ge.to(DEV), out=logits if in_place else None)
    terms = torch.exp(lp) * (gl.abs()[:, None] + ge.abs()[:, None] * (lp.clamp(min=-200).abs() + ref["entropy"][:, None]))
    want = ref["grad_logits"]
    bound = 8e-6 * (terms + want.abs()) + 1e-38 + (2.0 ** -8 * want.abs() if logits.dtype == torch.bfloat16 else 0)
    assert ((f64(out) - want).abs() <= bound).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [5, 1000, 20011])
@pytest.mark.parametrize("top", [0, 3])
def test_lowest_values(V, top, dtype):
    """Rows of nothing but the type's lowest value are uniform; one better value takes all."""
    low = torch.finfo(dtype).min
    x = torch.full((3, V), low, dtype=dtype)
    x[1, V - 2] = -1.0
    x[2, : V // 2] = -torch.inf
    target = torch.tensor([1, V - 2, V - 1])
    if top == 3 and V == 5:
        x[2, :] = low  # three finite alternatives
    run(x.to(DEV), target.to(DEV), top)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [-3e4, -300.0, 250.0, 300.0, 1e6])
@pytest.mark.parametrize("in_place", [False, True])
def test_shifted(shift, in_place, dtype):
    g = torch.Generator().manual_seed(5)
    N, V = 4, 40001
    x = (3 * torch.randn(N, V, generator=g) + shift).to(dtype)
    target = torch.randint(0, V, (N,), generator=g)
    target[2] = -100
    run(x.to(DEV), target.to(DEV), 0, in_place)
