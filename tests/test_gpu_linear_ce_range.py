"""Cross entropy of a linear head where the sizes of its values differ: classes that
are rare in every row, rows and features far larger than the others, rows without a
gradient that hold anything, against the plain fp64 form (lm_ref.py).

Bounds: those of test_gpu_linear_ce.py for an element of a gradient, relative to the
sum of the absolute terms of that element, so that a class whose probabilities are all
1e-8 is held to its own size.  bf16: 2^-8 of that sum (G rounded to 2^-8 at most, its
exponentials to 2^-11 down to 2^-29 of the largest of the classes around them), plus
2^-8 of the value.  fp32: 3e-5 of sum and value (the logits' rounding), plus what the
two parts leave of small values: half a unit of 2^-49 in G, next to any other factor,
and 2^-38 of the other factor's largest value, next to any element of G (G's scale is
2^14 and its low part's 2^25, the others' are at least 2^13 over the largest; fp16 ends
at 2^-24)."""
import numpy as np
import pytest
import torch

import linear_recurrence_scan_diagonal_amd as lrs
import lm_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def absolute_g(x, w, target):
    """Mean over the rows of |G| of each class."""
    logits = f64(x) @ f64(w).T
    with np.errstate(invalid="ignore"):
        p = np.exp(logits - logits.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
    t = target.cpu().numpy()
    rows = np.nonzero((t >= 0) & (t < len(w)))[0]
    p[rows, t[rows]] -= 1.0
    return np.abs(p[rows]).sum(0) / len(x)


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
    tol, least, other = (3e-5, 2.0 ** -49, 2.0 ** -38) if f32 else (2.0 ** -8, 0.0, 0.0)
    counts = ((target >= 0) & (target < len(w))).cpu().numpy()
    g = np.abs(f64(gl)) * counts
    ax, aw = np.abs(f64(x)) * (g > 0)[:, None], np.abs(f64(w))
    top_x, top_w = (ax * g[:, None]).max(initial=0.0), aw.max()
    # a row's |G| sums to 2 at most; a class's to the number of rows
    floor = {"grad_x": (least * len(w) + 2 * other + slack) * g[:, None] * top_w,
             "grad_w": ((least + other * absolute_g(x, w, target)[:, None]) * len(x) + slack) * top_x}
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


@BOTH
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


@BOTH
@pytest.mark.parametrize("size", [3.0, 1e4])
def test_rows_do_not_depend_on_their_neighbours(dtype, size):
    """Loss, lse and gradient of a row have the same bits next to rows of any size."""
    g = torch.Generator().manual_seed(10)
    N, V, D = 80, 300, 64
    x, w = torch.randn(N, D, generator=g).to(dtype).to(DEV), torch.randn(V, D, generator=g).to(dtype).to(DEV)
    target, gl = torch.arange(N, device=DEV), torch.full((N,), 1.0 / N, device=DEV)
    want = lrs.linear_ce_fwd_bwd(x, w, target, gl)
    x2, own = x.clone(), torch.arange(N, device=DEV) % 5 != 0
    x2[~own] *= size
    got = lrs.linear_ce_fwd_bwd(x2, w, target, gl)
    assert all(torch.equal(a[own], b[own]) for a, b in zip(got[:3], want))


@BOTH
@pytest.mark.parametrize("value", [float("inf"), float("nan"), 1e12, -1e30])
def test_rows_without_a_gradient_hold_anything(dtype, value):
    """A row that counts, with a grad_loss of 0, changes no other row's gradient and
    nothing of grad_w, whatever it holds."""
    g = torch.Generator().manual_seed(6)
    N, V, D = 90, 260, 64
    x, w = torch.randn(N, D, generator=g).to(dtype).to(DEV), torch.randn(V, D, generator=g).to(dtype).to(DEV)
    target = torch.arange(N, device=DEV)
    gl = torch.full((N,), 0.5, device=DEV)
    gl[11] = gl[60] = 0.0
    want = lrs.linear_ce_fwd_bwd(x, w, target, gl)
    x2 = x.clone()
    x2[11, 3] = value
    x2[60] = value
    got = lrs.linear_ce_fwd_bwd(x2, w, target, gl)
    assert torch.equal(got[2], want[2]) and torch.equal(got[3], want[3])
    lse = lrs.linear_ce_fwd(x2, w, target)[1]
    assert all(torch.equal(a, b) for a, b in zip(lrs.linear_ce_bwd(x2, w, target, lse, gl), want[2:]))
    check(x, w, target, gl)


@BOTH
def test_large_rows_with_a_small_share(dtype):
    """A row 1e9 times as large whose loss weighs 1e-12: its part of grad_w is small,
    and the other rows' parts keep their digits."""
    g = torch.Generator().manual_seed(7)
    N, V, D = 120, 200, 40
    x, w = torch.randn(N, D, generator=g), 0.2 * torch.randn(V, D, generator=g)
    gl = torch.full((N,), 0.01)
    x[17] *= 1e9
    gl[17] = 1e-14
    check(*(t.to(DEV) for t in (x.to(dtype), w.to(dtype), torch.arange(N), gl)))


@BOTH
def test_an_outlier_feature(dtype):
    """A class with a weight of 1e3 in a feature that x has little of: the other classes'
    parts of grad_x keep their digits."""
    g = torch.Generator().manual_seed(8)
    N, V, D = 130, 300, 48
    x, w = torch.randn(N, D, generator=g), 0.2 * torch.randn(V, D, generator=g)
    x[:, 5] *= 1e-3
    w[33, 5] = 1e3
    check(*(t.to(DEV) for t in (x.to(dtype), w.to(dtype), torch.randint(0, V, (N,), generator=g),
                                torch.full((N,), 1.0 / N))))


@BOTH
@pytest.mark.parametrize("V,D", [(30, 16), (7, 3), (1, 1), (1, 2), (3000, 501)])
@pytest.mark.parametrize("shift", [0, 1, 2, 3])
def test_no_rows_any_alignment(dtype, V, D, shift):
    """Without rows grad_w is 0, to its first and last element and not past them,
    wherever it begins."""
    x, target, gl = (torch.empty(0, D, dtype=dtype, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV),
                     torch.empty(0, device=DEV))
    wide = torch.full((V * D + 8,), 7.0, dtype=dtype, device=DEV)
    gw = wide[shift:shift + V * D].view(V, D)
    lrs.linear_ce_fwd_bwd(x, torch.ones(V, D, dtype=dtype, device=DEV), target, gl, out=(x.clone(), gw))
    assert (gw == 0).all() and (wide[:shift] == 7).all() and (wide[shift + V * D:] == 7).all()


@pytest.mark.parametrize("N,V,D,dtype", [(16384, 32768, 1024, torch.bfloat16), (4099, 50021, 777, torch.bfloat16),
                                         (2048, 16384, 512, torch.float32), (40000, 40000, 72, torch.bfloat16)])
def test_large_calls_repeat_themselves(N, V, D, dtype):
    """Thousands of tiles, shares of the k loop and pieces of rows: the same bits from
    call to call, from whatever the workspace held before."""
    g = torch.Generator(device=DEV).manual_seed(N)
    x = torch.randn(N, D, generator=g, device=DEV).to(dtype)
    w = (torch.randn(V, D, generator=g, device=DEV) * 2 / D ** 0.5).to(dtype)
    target = torch.randint(-V // 20, V, (N,), generator=g, device=DEV)
    gl = torch.full((N,), 1.0 / N, device=DEV)
    nbytes = lrs.load().lrs_linear_ce_workspace_bytes(N, V, D, int(dtype == torch.bfloat16), 1)
    runs = []
    for fill in (0, 255, 60, 127):
        ws = torch.full((nbytes,), fill, dtype=torch.uint8, device=DEV)
        runs.append(lrs.linear_ce_fwd_bwd(x, w, target, gl, workspace=ws))
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(runs[0], r))
