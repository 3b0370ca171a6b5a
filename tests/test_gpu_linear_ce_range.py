"""Cross entropy of a linear head where the sizes of its values differ: classes that
are rare in every row, rows and features far larger than the others, rows without a
gradient that hold anything, against the plain fp64 form (lm_ref.py).

Bounds: those of test_gpu_linear_ce.py for an element of a gradient, relative to the
sum of the absolute terms of that element, so that a class whose probabilities are all
1e-8 is held to its own size.  bf16: 2^-8 of that sum (G rounded to 2^-8 at most, its
exponentials to 2^-11 down to 2^-29 of the largest of the classes around them), plus
2^-8 of the value.  fp32: 3e-5 of sum and value (the logits' rounding), plus what the
two parts leave of small values: 2^-50 in G and 2^-49 of the other factor's largest
value, at most 2^-48 of the largest term in each of the sum's terms."""
import numpy as np
import pytest
import torch

import linear_recurrence_scan_diagonal_amd as lrs
import lm_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
BF16 = pytest.mark.parametrize("dtype", [torch.bfloat16])


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def check(x, w, target, gl, slack=0.0):
    """Both ways to the gradient; returns the plain form's results.  slack: an absolute
    error of G (a multiple of grad_loss) that the bound leaves besides."""
    loss, lse = lrs.linear_ce_fwd(x, w, target)
    apart = lrs.linear_ce_bwd(x, w, target, lse, gl)
    both = lrs.linear_ce_fwd_bwd(x, w, target, gl)
    torch.cuda.synchronize()
    ref = R.linear_ce(f64(x), f64(w), target.cpu().numpy(), f64(gl))
    for l, s in ((loss, lse), both[:2]):
        for name, t in (("loss", l), ("lse", s)):
            off = np.abs(f64(t) - ref[name]) / (1 + np.abs(ref[name]))
            assert off.max() <= 1e-5, (name, off.max())
    f32 = x.dtype == torch.float32
    tol, least = (3e-5, 2.0 ** -48) if f32 else (2.0 ** -8, 0.0)
    counts = ((target >= 0) & (target < len(w))).cpu().numpy()
    g = np.abs(f64(gl)) * counts
    # the largest term there could be: a whole row's probability times the largest factor
    ax, aw = np.abs(f64(x)) * (g > 0)[:, None], np.abs(f64(w))
    top_x, top_w = (ax * g[:, None]).max(initial=0.0), aw.max()
    floor = {"grad_x": (least * len(w) + slack) * g[:, None] * top_w,
             "grad_w": (least * len(x) + slack) * top_x}
    for gx, gw in (apart, both[2:]):
        for name, t in (("grad_x", gx), ("grad_w", gw)):
            r, s = ref[name], ref["scale_" + name]
            off = np.abs(f64(t) - r) - tol * (s + np.abs(r)) - floor[name]
            assert np.isfinite(f64(t)).all() and off.max() <= 1e-38, (name, off.max())
    return ref


def rare(N, V, D, dtype, nats, seed, spread=0.15):
    """The second half of the classes lie `nats` below the first in every row; targets
    are of the first half."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, w = n(N, D), n(V, D) * spread / D ** 0.5
    x[:, 0], w[:, 0] = 1.0, 0.0
    w[V // 2:, 0] = -nats
    w = w[torch.randperm(V, generator=g)]
    common = torch.nonzero(w[:, 0] == 0.0)[:, 0]
    target = common[torch.randint(0, len(common), (N,), generator=g)]
    gl = torch.full((N,), 1.0 / N)
    return [t.to(DEV) for t in (x.to(dtype), w.to(dtype), target, gl)]


@BF16
@pytest.mark.parametrize("N,V,D", [(100, 300, 32), (512, 1024, 64), (700, 12000, 72), (1300, 40960, 64)])
@pytest.mark.parametrize("nats", [8.0, 13.0, 17.5])
def test_rare_classes(N, V, D, dtype, nats):
    """A class that is improbable in every row keeps the digits of its gradient."""
    x, w, target, gl = rare(N, V, D, dtype, nats, N)
    logits = f64(x) @ f64(w).T
    # all inside the range in which the bounds hold (20 nats: 2^-29)
    assert logits.max() - logits.min() < 20.0
    check(x, w, target, gl)


@BOTH
def test_rows_that_are_certain(dtype):
    """Targets of probability 1 - 3e-5: p - 1 is what fp32 logits and lse of size 16 leave
    of it (one unit in the last place each, 4e-6 together), not more."""
    g = torch.Generator().manual_seed(5)
    N = V = 256
    x = torch.eye(N)
    w = 16.0 * torch.eye(V) + 0.1 * torch.randn(V, V, generator=g)
    x, w = x.to(dtype).to(DEV), w.to(dtype).to(DEV)
    check(x, w, torch.arange(N, device=DEV), torch.full((N,), 1.0 / N, device=DEV), slack=4e-6)


@BOTH
def test_large_logits(dtype):
    """Rows whose largest logit is 1 to 1000, next to each other.  A logit's rounding,
    1e-6 of its absolute sum (some 2000 at most), is a relative error of G."""
    g = torch.Generator().manual_seed(9)
    N, V, D = 150, 700, 40
    x, w = torch.randn(N, D, generator=g), torch.randn(V, D, generator=g)
    x *= torch.logspace(-1.5, 1.5, N)[torch.randperm(N, generator=g)][:, None]
    x, w = x.to(dtype), w.to(dtype)
    logits = f64(x) @ f64(w).T
    assert logits.max() > 500 and logits.max(1).min() < 2
    check(x.to(DEV), w.to(DEV), torch.randint(0, V, (N,), generator=g).to(DEV),
          torch.full((N,), 1.0 / N, device=DEV), slack=4e-3)
