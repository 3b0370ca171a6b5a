"""The fp64 forms in lm_ref.py against automatic differentiation and central
differences, and their statements about masked rows."""
import numpy as np
import pytest
import torch

import lm_ref as R


def _torch_glr(zr, zi, x, br, bi, decay, c, reset, h0, gh, gl):
    r, i = torch.sigmoid(zr + br), torch.sigmoid(zi + bi)
    la = -c * torch.nn.functional.softplus(decay) * r
    h, s = h0, 0.0
    for t in range(zr.shape[0]):
        keep = (reset[t] == 0).double()[:, None]
        a = torch.exp(la[t]) * keep
        m = torch.where(keep > 0, torch.sqrt(-torch.expm1(2 * la[t])), torch.ones_like(la[t]))
        h = a * h + m * i[t] * x[t]
        s = s + (h * gh[t]).sum()
    return s + (h * gl).sum()


@pytest.mark.parametrize("T,B,D", [(1, 1, 1), (7, 2, 3), (19, 1, 5)])
def test_glr_gradient_against_autograd_and_differences(T, B, D):
    rng = np.random.default_rng(T)
    zr, zi, x, gh = (rng.normal(size=(T, B, D)) for _ in range(4))
    br, bi, decay = rng.normal(size=D), rng.normal(size=D), rng.normal(-2, 1, D)
    h0, gl = rng.normal(size=(B, D)), rng.normal(size=(B, D))
    reset = (rng.random((T, B)) < 0.2).astype(np.uint8)
    got = R.glr(zr, zi, x, br, bi, decay, 8.0, reset, h0, gh, gl)
    leaf = [torch.tensor(v, requires_grad=True) for v in (zr, zi, x, br, bi, decay, h0)]
    loss = _torch_glr(*leaf[:6], 8.0, torch.tensor(reset), leaf[6], torch.tensor(gh),
                      torch.tensor(gl))
    loss.backward()
    names = ("grad_zr", "grad_zi", "grad_x", "grad_bias_r", "grad_bias_i", "grad_decay", "grad_h0")
    for name, t in zip(names, leaf):
        np.testing.assert_allclose(got[name], t.grad.numpy(), rtol=1e-9, atol=1e-11, err_msg=name)

    def value(d):
        o = R.glr(zr, zi, x, br, bi, decay + d, 8.0, reset, h0)
        return (o["h"] * gh).sum() + (o["h_last"] * gl).sum()
    e = 1e-5
    diff = (value(e) - value(-e)) / (2 * e)
    # central differences: error e^2 times a third derivative, and 1e-16 / e of rounding
    assert abs(diff - got["grad_decay"].sum()) <= 1e-6 * (1 + got["scale_grad_decay"].sum())


def test_glr_reset_cuts_everything():
    rng = np.random.default_rng(0)
    T, B, D = 6, 1, 2
    z = [rng.normal(size=(T, B, D)) for _ in range(4)]
    reset = np.zeros((T, B), np.uint8)
    reset[3] = 1
    p = [rng.normal(size=D) for _ in range(3)]
    bad = z[2].copy()
    bad[1] = np.nan
    out = R.glr(z[0], z[1], bad, *p, 8.0, reset, None, z[3])
    assert np.isnan(out["h"][1:3]).all() and np.isfinite(out["h"][3:]).all()
    assert np.isfinite(out["grad_x"][3:]).all() and (out["grad_zr"][3] == 0).all()


def test_layernorm_gradient():
    rng = np.random.default_rng(1)
    s, gy = rng.normal(size=(5, 7)), rng.normal(size=(5, 7))
    gamma, beta = rng.normal(size=7), rng.normal(size=7)
    got = R.layernorm(s, gamma, beta, 1e-5, gy)
    ts, tg, tb = (torch.tensor(v, requires_grad=True) for v in (s, gamma, beta))
    y = torch.nn.functional.layer_norm(ts, (7,), tg, tb, 1e-5)
    (y * torch.tensor(gy)).sum().backward()
    for name, t in (("grad_x", ts), ("grad_gamma", tg), ("grad_beta", tb)):
        np.testing.assert_allclose(got[name], t.grad.numpy(), rtol=1e-9, atol=1e-11)


def test_linear_ce_gradient():
    rng = np.random.default_rng(2)
    x, w, gl = rng.normal(size=(6, 4)), rng.normal(size=(9, 4)), rng.normal(size=6)
    target = np.array([0, 8, -100, 3, 9, 2])
    got = R.linear_ce(x, w, target, gl)
    tx, tw = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    t = torch.tensor(np.where(target == 9, -100, target))
    loss = torch.nn.functional.cross_entropy(tx @ tw.t(), t, reduction="none", ignore_index=-100)
    np.testing.assert_allclose(got["loss"], loss.detach().numpy(), rtol=1e-12, atol=1e-12)
    (loss * torch.tensor(gl)).sum().backward()
    np.testing.assert_allclose(got["grad_x"], tx.grad.numpy(), rtol=1e-9, atol=1e-12)
    np.testing.assert_allclose(got["grad_w"], tw.grad.numpy(), rtol=1e-9, atol=1e-12)
