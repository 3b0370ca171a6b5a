"""Gates and memories of the gated linear recurrence over their whole range, in both
plans, against the plain fp64 form (lm_ref.py).

The exponent of an open gate is k = c softplus(decay).  A wave whose channels all
have k < 1/8 takes a shorter form of a = exp(-k r) and sqrt(1 - a^2), every other wave
the general one.  The bounds are those of test_gpu_glr.py, whose roundings both forms
share: 1e-5 of 1 + |value|, plus 2^-8 of the value in bf16; the parameters' gradients
1e-5 of the sum of the absolute terms."""
import numpy as np
import pytest
import torch

import linear_recurrence_scan_diagonal_amd as lrs
import lm_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = {torch.float32: 1e-5, torch.bfloat16: 2.0 ** -8 + 1e-5}
NAMES = ("grad_zr", "grad_zi", "grad_x", "grad_bias_r", "grad_bias_i", "grad_decay", "grad_h0")
SIZES = {"tiles": (300, 2, 130), "odd tiles": (77, 3, 35), "walk": (150, 65, 512),
         "odd walk": (131, 64, 521)}


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def check(parts, p, reset, h0, gh, gl):
    dtype = parts[0].dtype
    ck = lrs.glr_checkpoints(parts[0])
    h, last = lrs.glr_fwd(*parts, **p, reset=reset, h0=h0, want_h_last=True, checkpoints=ck)
    grads = lrs.glr_bwd(*parts, **p, checkpoints=ck, grad_h=gh, reset=reset, grad_h_last=gl)
    torch.cuda.synchronize()
    ref = R.glr(*(f64(t) for t in parts), f64(p["bias_r"]), f64(p["bias_i"]), f64(p["decay"]), 8.0,
                None if reset is None else reset.cpu().numpy(), f64(h0), f64(gh), f64(gl))
    for name, t in {"h": h, "h_last": last, **dict(zip(NAMES, grads))}.items():
        t, want = f64(t), ref[name]
        own = ref.get("scale_" + name)
        off = np.abs(t - want) / (1 + np.abs(want if own is None else own))
        assert off.max() <= (TOL[dtype] if t.ndim == 3 else 1e-5), (name, off.max())
    return h, grads


def make(T, B, D, dtype, seed, decay):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    parts = [n(T, B, D).to(dtype).to(DEV) for _ in range(3)]
    p = {"bias_r": 0.3 * n(D), "bias_i": 0.3 * n(D), "decay": decay(D)}
    rest = [n(B, D), n(T, B, D).to(dtype), n(B, D)]
    return parts, {k: v.to(DEV) for k, v in p.items()}, [v.to(DEV) for v in rest]


# k between: 0.02 and 0.1 (the short form), 0.25 and 24 (the general one), both in one wave
DECAYS = {"long": lambda D: torch.linspace(-6.0, -4.4, D), "short": lambda D: torch.linspace(-3.4, 3.0, D),
          "mixed": lambda D: torch.linspace(-6.0, 3.0, D)[torch.randperm(D, generator=torch.Generator().manual_seed(1))]}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("memory", DECAYS)
@pytest.mark.parametrize("restart", [0.0, 0.03])
def test_memories(size, dtype, memory, restart):
    T, B, D = SIZES[size]
    parts, p, rest = make(T, B, D, dtype, T + D, DECAYS[memory])
    reset = None
    if restart:
        g = torch.Generator().manual_seed(T)
        reset = (torch.rand(T, B, generator=g) < restart).to(torch.uint8).to(DEV)
    check(parts, p, reset, *rest)


def test_the_border_of_the_two_forms():
    """k a hair below and above 1/8: no step between the forms."""
    T, B, D = 200, 2, 128
    border = float(np.log(np.expm1(1.0 / 64.0)))  # 8 softplus = 1/8
    for seed, side in enumerate((-1e-4, 1e-4)):
        parts, p, rest = make(T, B, D, torch.float32, seed, lambda D: torch.full((D,), border + side))
        check(parts, p, None, *rest)


def test_parameter_gradients_of_a_long_walk():
    """40000 steps of constant inputs, 32768 channels: every term of a parameter's
    gradient has the same sign and nearly the same value, so a running fp32 sum would
    lose up to 1e-4 of it.  All 512 sequences are alike."""
    T, B, D = 40_000, 512, 64
    g = torch.Generator().manual_seed(0)
    rows = [(torch.randn(D, generator=g).abs() + 0.25).bfloat16() for _ in range(4)]  # z_r, z_i, x, grad_h
    p = {"bias_r": 0.3 * torch.randn(D, generator=g), "bias_i": 0.3 * torch.randn(D, generator=g),
         "decay": torch.linspace(-4.0, 0.0, D)}
    one = [f64(v)[None, None].repeat(T, 0) for v in rows]
    ref = R.glr(*one[:3], *(f64(v) for v in p.values()), 8.0, gh=one[3])
    zr, zi, x, gh = (v.to(DEV).expand(T, B, D).contiguous() for v in rows)
    p = {k: v.to(DEV) for k, v in p.items()}
    ck = lrs.glr_checkpoints(zr)
    lrs.glr_fwd(zr, zi, x, **p, checkpoints=ck)
    grads = lrs.glr_bwd(zr, zi, x, **p, checkpoints=ck, grad_h=gh)
    for name, t in list(zip(NAMES, grads))[3:6]:
        off = np.abs(f64(t) / B - ref[name]) / ref["scale_" + name]
        assert off.max() <= 1e-5, (name, off.max())


@pytest.mark.parametrize("size", SIZES)
def test_closed_gates_with_large_inputs(size):
    """A gate closed to the last bit has a = 1 and m = 0: nothing of x enters, however
    large, and the terms with 1/m are 0."""
    T, B, D = SIZES[size]
    parts, p, rest = make(T, B, D, torch.float32, 3, DECAYS["mixed"])
    parts[0][:, :, ::2] = -300.0
    parts[2][:, :, ::2] = 1e20
    h, grads = check(parts, p, None, *rest)
    for t in (grads[0], grads[1], grads[2]):
        assert (t[:, :, ::2] == 0).all()
    assert torch.equal(h[-1, :, ::2], rest[0][:, ::2])


@pytest.mark.parametrize("size", SIZES)
def test_memories_without_an_end(size):
    """softplus(decay) rounds to 0: a = 1, m = 0 and a zero gradient of decay, whatever
    the gate is."""
    T, B, D = SIZES[size]
    parts, p, rest = make(T, B, D, torch.float32, 4, lambda D: torch.full((D,), -300.0))
    parts[2] *= 1e12
    h, grads = check(parts, p, None, *rest)
    assert (grads[0] == 0).all() and (grads[5] == 0).all()
