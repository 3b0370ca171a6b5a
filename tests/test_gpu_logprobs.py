"""Log probabilities of given tokens, entropy and the likeliest alternatives on the GPU
against the plain fp64 form.

Bounds.  An exponential's argument is off by its rounding, 2^-24 of a difference of up to
the logits' spread, and the logarithm by 6e-8 of itself: 2e-6 of 1 + |value| for spreads of
up to 30.  The gradient takes lse as it was rounded, 2^-24 |lse|: 4e-6 of a probability,
with |lse| + spread at most 60, plus the rounding to the output's type (bf16 2^-8)."""
import math

import pytest
import torch

import linear_recurrence_scan_diagonal_amd as lrs
import block_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def f64(t):
    return t.detach().cpu().double()


def make(N, V, dtype=torch.float32, seed=0, spread=3.0, ignored=0.2):
    g = torch.Generator().manual_seed(seed)
    logits = (spread * torch.randn(N, V, generator=g)).to(dtype)
    target = torch.randint(0, V, (N,), generator=g)
    target = torch.where(torch.rand(N, generator=g) < ignored, torch.where(torch.rand(N, generator=g) < 0.5, -100, V), target)
    return logits.to(DEV), target.to(DEV)


def close(name, got, ref, tol):
    off = (f64(got) - ref).abs() / (1.0 + ref.abs())
    off = torch.where(f64(got) == ref, 0.0, off)  # infinities that agree
    assert off.max() <= tol, (name, float(off.max()))


def check(logits, target, top=0, grads=True, seed=1):
    N, V = logits.shape
    logprob, entropy, lse, ids, tops = lrs.logprobs_fwd(logits, target, top=top)
    g = torch.Generator().manual_seed(seed)
    gl, ge = torch.randn(N, generator=g), torch.randn(N, generator=g)
    ref = R.logprobs(f64(logits), target.cpu(), gl.double(), ge.double())
    for name, got in (("logprob", logprob), ("entropy", entropy), ("lse", lse)):
        close(name, got, ref[name], 2e-6)
    assert (logprob[(target < 0) | (target >= V)] == 0).all()
    if top:
        want = R.tops(f64(logits), top)
        assert torch.equal(ids.cpu(), want)
        close("tops", tops, ref["lp"].gather(1, want), 2e-6)
    else:
        assert ids is None and tops is None
    if grads:
        for e in (None, ge):
            out = lrs.logprobs_bwd(logits, target, lse, entropy, gl.to(DEV), None if e is None else e.to(DEV))
            want = R.logprobs(f64(logits), target.cpu(), gl.double(), None if e is None else e.double())["grad_logits"]
            p = torch.exp(ref["lp"])
            terms = p * (gl.abs()[:, None] + (0 if e is None else e.abs()[:, None] * (ref["lp"].clamp(min=-200).abs() + ref["entropy"][:, None])))
            bound = 8e-6 * (terms + want.abs()) + 1e-38 + (2.0 ** -8 * want.abs() if logits.dtype == torch.bfloat16 else 0)
            assert ((f64(out) - want).abs() <= bound).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,V,top", [(1, 1, 1), (3, 2, 2), (5, 7, 7), (2, 63, 1), (9, 64, 64), (4, 100, 33), (3, 1000, 5),
                                     (7, 4097, 20), (2, 8191, 32), (5, 8192, 64), (3, 16400, 8), (4, 32000, 50),
                                     (2, 33333, 10), (3, 65537, 20), (2, 131072, 20), (2, 131073, 64), (1, 300001, 7)])
def test_parity(N, V, top, dtype):
    check(*make(N, V, dtype, seed=N + V), top=top)
    check(*make(N, V, dtype, seed=N + V + 1), top=0, grads=False)


@pytest.mark.parametrize("top", [1, 8, 64])
@pytest.mark.parametrize("how", ["equal", "two values", "rising", "falling", "blocks", "zeros of both signs", "few finite"])
def test_order(how, top):
    """Ties go to the lower index; any order along the row."""
    N, V = 3, 5000
    x = torch.zeros(N, V)
    g = torch.Generator().manual_seed(2)
    if how == "two values":
        x = (torch.rand(N, V, generator=g) < 0.5).float()
    elif how in ("rising", "falling"):
        x = torch.arange(V).float().expand(N, V) * (1e-3 if how == "rising" else -1e-3)
    elif how == "blocks":  # everything large within what one thread reads
        x = torch.randn(N, V, generator=g)
        x[:, 2048:2056] += 20
        x[:, 0:8] += 10
        x[:, 4096:4100] += 30
    elif how == "zeros of both signs":
        x = torch.where(torch.rand(N, V, generator=g) < 0.5, 0.0, -0.0)
    elif how == "few finite":
        x = torch.full((N, V), -math.inf)
        x[:, [17, 4000, 4999]] = torch.tensor([1.0, 3.0, 1.0])
    x = x.contiguous().to(DEV)
    target = torch.tensor([17, 0, -1], device=DEV)
    if how == "few finite":
        target[1] = 4000
    check(x, target, top=top)
    check(x.bfloat16(), target, top=top)


@pytest.mark.parametrize("V", [1000, 33333, 300001])
def test_order_of_wide_rows_with_ties(V):
    x = torch.randint(0, 3, (2, V), generator=torch.Generator().manual_seed(3)).float().to(DEV)
    check(x, torch.tensor([5, 6], device=DEV), top=64, grads=False)


def test_masked_logits():
    """-infinity (a token that may not follow) adds nothing, has probability 0 and gradient 0."""
    logits, target = make(20, 3001, seed=4)
    logits[:, 1::2] = -math.inf
    logits[3, 1:] = -math.inf  # one token left: entropy 0
    target[:] = 0
    check(logits, target, top=5)
    _, entropy, lse, _, _ = lrs.logprobs_fwd(logits, target)
    assert entropy[3] == 0
    g = lrs.logprobs_bwd(logits, target, lse, entropy, torch.ones(20, device=DEV), torch.ones(20, device=DEV))
    assert (g[:, 1::2] == 0).all()
    low = torch.full((2, 100), torch.finfo(torch.float32).min, device=DEV)  # the type's lowest value as a mask
    low[:, 7] = 1.0
    check(low, torch.tensor([7, 7], device=DEV), top=3)


@pytest.mark.parametrize("V", [100, 20000, 300000])
def test_rows_without_probabilities(V):
    logits, target = make(6, V, seed=5, ignored=0)
    clean = lrs.logprobs_fwd(logits, target, top=3)
    logits[1] = -math.inf
    logits[2, V // 2] = math.nan
    logits[4, V - 1] = math.inf
    out = lrs.logprobs_fwd(logits, target, top=3)
    logprob, entropy, lse, ids, tops = out
    for r in (1, 2, 4):
        assert torch.isnan(logprob[r]) and torch.isnan(entropy[r]) and torch.isnan(tops[r]).all()
    assert lse[1] == -math.inf and torch.isnan(lse[2]) and lse[4] == math.inf
    assert ids[1].tolist() == [0, 1, 2] and ids[2, 0] == V // 2 and ids[4, 0] == V - 1
    assert torch.equal(ids.cpu(), R.tops(logits.cpu().double().nan_to_num(posinf=1e300, neginf=-1e300, nan=math.nan), 3))
    keep = [0, 3, 5]
    for a, b in zip(out, clean):
        assert torch.equal(a[keep], b[keep])


def test_ignored_rows():
    """A padded row asks for nothing: its gradient is 0 whatever its logits hold."""
    logits, target = make(5, 999, seed=6, ignored=0)
    target[2] = -100
    logits[2] = math.nan
    logprob, entropy, lse, _, _ = lrs.logprobs_fwd(logits, target)
    assert logprob[2] == 0
    ones = torch.ones(5, device=DEV)
    g = lrs.logprobs_bwd(logits, target, lse, entropy, ones)
    assert (g[2] == 0).all() and torch.isfinite(g).all()
    ge = ones.clone()
    ge[2] = 0
    g = lrs.logprobs_bwd(logits, target, lse, entropy, ones, ge)
    assert (g[2] == 0).all() and torch.isfinite(g).all()


def test_certain_token():
    """A token that is nearly certain: its log probability is -sum of the others, not 0."""
    logits = torch.full((1, 1000), -10.0, device=DEV)
    logits[0, 3] = 0.0
    check(logits, torch.tensor([3], device=DEV), top=2)
    lp = lrs.logprobs_fwd(logits, torch.tensor([3], device=DEV))[0]
    want = -math.log1p(999 * math.exp(-10))
    assert abs(float(lp) - want) < 2e-7  # one rounding of 1 + 0.045


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_padded_rows_and_in_place(dtype):
    """Rows that are slices of wider ones, at an odd pitch; the gradient over the logits."""
    logits, target = make(9, 1003, dtype, seed=7)
    wide = torch.full((9, 1111), math.nan, dtype=dtype, device=DEV)
    view = wide[:, 5:1008]
    view.copy_(logits)
    want, got = lrs.logprobs_fwd(logits, target, top=9), lrs.logprobs_fwd(view, target, top=9)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    gl = torch.randn(9, device=DEV)
    g = lrs.logprobs_bwd(logits, target, want[2], want[1], gl, gl)
    out = torch.full((9, 1200), 7.0, dtype=dtype, device=DEV)
    lrs.logprobs_bwd(view, target, want[2], want[1], gl, gl, out=out[:, 1:1004])
    assert torch.equal(out[:, 1:1004], g) and (out[:, 1004:] == 7).all() and (out[:, 0] == 7).all()
    lrs.logprobs_bwd(view, target, want[2], want[1], gl, gl, out=view)
    assert torch.equal(view, g) and torch.isnan(wide[:, :5].float()).all() and torch.isnan(wide[:, 1008:].float()).all()


def test_gradient_against_differences():
    logits, target = make(5, 203, seed=8, ignored=0)
    logprob, entropy, lse, _, _ = lrs.logprobs_fwd(logits, target)
    gen = torch.Generator().manual_seed(1)
    gl, ge, d = torch.randn(5, generator=gen), torch.randn(5, generator=gen), torch.randn(5, 203, generator=gen).double()
    g = f64(lrs.logprobs_bwd(logits, target, lse, entropy, gl.to(DEV), ge.to(DEV)))

    def f(h):
        r = R.logprobs(f64(logits) + h * d, target.cpu())
        return (r["logprob"] * gl.double() + r["entropy"] * ge.double()).sum()
    slope = (f(1e-5) - f(-1e-5)) / 2e-5
    assert abs((g * d).sum() - slope) <= 1e-5 * (g * d).abs().sum()


def test_empty():
    logits = torch.empty(0, 50, device=DEV)
    out = lrs.logprobs_fwd(logits, torch.empty(0, dtype=torch.int64, device=DEV), top=3)
    assert out[0].shape == (0,) and out[3].shape == (0, 3)
    e = torch.empty(0, device=DEV)
    assert lrs.logprobs_bwd(logits, torch.empty(0, dtype=torch.int64, device=DEV), e, e, e).shape == (0, 50)


def test_refusals():
    logits, target = make(4, 50)
    with pytest.raises(TypeError):
        lrs.logprobs_fwd(logits.half(), target)
    with pytest.raises(TypeError):
        lrs.logprobs_fwd(logits, target.int())
    with pytest.raises(ValueError):
        lrs.logprobs_fwd(logits.t(), target)
    with pytest.raises(ValueError):
        lrs.logprobs_fwd(logits, target, top=51)
    with pytest.raises(ValueError):
        lrs.logprobs_fwd(logits.repeat(1, 2), target, top=65)
    with pytest.raises(ValueError):
        lrs.logprobs_fwd(logits, target, top=-1)
    e = torch.zeros(4, device=DEV)
    with pytest.raises(TypeError):
        lrs.logprobs_bwd(logits, target, e, None, e, e)
    with pytest.raises(TypeError):
        lrs.logprobs_bwd(logits, target, None, e, e)
    with pytest.raises(lrs.LrsError):  # shifted over the logits
        wide = torch.zeros(4, 60, device=DEV)
        lrs.logprobs_bwd(wide[:, :50], target, e, e, e, out=wide[:, 1:51])
    with pytest.raises(ValueError):
        lrs.logprobs_fwd(torch.zeros(4, 0, device=DEV), target, top=1)
