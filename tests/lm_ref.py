"""Plain fp64 forms of the language-model operators (include/lrs_lm.h): one time
step, one row or one product after the other, on the CPU, sharing no code with
the device path."""
import numpy as np


def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def softplus(v):
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def glr(zr, zi, x, br, bi, decay, c, reset=None, h0=None, gh=None, gh_last=None):
    """Forward, and with gh the gradients, of the gated linear recurrence on
    [T,B,D] float64 arrays.  Returns a dict; "scale_*" are sums of the absolute
    terms of the parameter gradients, which bound what rounding can do to them."""
    T, B, D = zr.shape
    h0 = np.zeros((B, D)) if h0 is None else h0
    r, i = sigmoid(zr + br), sigmoid(zi + bi)
    la = -c * softplus(decay) * r
    a, m = np.exp(la), np.sqrt(-np.expm1(2.0 * la))
    cut = np.zeros((T, B), dtype=bool) if reset is None else np.asarray(reset) != 0
    h, before = np.empty_like(zr), np.empty_like(zr)
    state = h0
    for t in range(T):
        a[t][cut[t]], m[t][cut[t]] = 0.0, 1.0
        # a restart drops the state, whatever it holds
        state = np.where(cut[t][:, None], 0.0, state)
        before[t] = state
        state = a[t] * state + m[t] * i[t] * x[t]
        h[t] = state
    out = {"h": h, "h_last": state if T else h0}
    if gh is None:
        return out
    lam = np.empty_like(h)
    carry = np.zeros((B, D)) if gh_last is None else gh_last
    for t in range(T - 1, -1, -1):
        lam[t] = gh[t] + carry
        carry = np.where(cut[t][:, None], 0.0, a[t] * lam[t])
    u = i * x
    with np.errstate(divide="ignore", invalid="ignore"):
        inv = np.where(m > 0.0, 1.0 / m, 0.0)
    dla = np.where(cut[..., None], 0.0, lam * (a * before - a * a * inv * u))
    dzr, dzi = dla * la * (1.0 - r), lam * m * x * i * (1.0 - i)
    dd = dla * r * (-c * sigmoid(decay))
    out.update(grad_zr=dzr, grad_zi=dzi, grad_x=lam * m * i, grad_h0=carry)
    for name, terms in (("grad_bias_r", dzr), ("grad_bias_i", dzi), ("grad_decay", dd)):
        out[name] = terms.sum((0, 1))
        out["scale_" + name] = np.abs(terms).sum((0, 1))
    return out


def layernorm(s, gamma, beta, eps, gy=None, gsum=None):
    mean = s.mean(1, keepdims=True)
    c = s - mean
    rstd = 1.0 / np.sqrt((c * c).mean(1, keepdims=True) + eps)
    xh = c * rstd
    out = {"y": xh * gamma + (0.0 if beta is None else beta), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if gy is None:
        return out
    q = gy * gamma
    dx = rstd * (q - q.mean(1, keepdims=True) - xh * (q * xh).mean(1, keepdims=True))
    out["grad_x"] = dx if gsum is None else dx + gsum
    out["grad_gamma"], out["grad_beta"] = (gy * xh).sum(0), gy.sum(0)
    out["scale_grad_gamma"], out["scale_grad_beta"] = np.abs(gy * xh).sum(0), np.abs(gy).sum(0)
    return out


def linear_ce(x, w, target, gl=None):
    """x [N,D], w [V,D] float64, target [N] ints."""
    V = w.shape[0]
    logits = x @ w.T
    top = logits.max(1)
    lse = top + np.log(np.exp(logits - top[:, None]).sum(1))
    counts = (target >= 0) & (target < V)
    rows = np.nonzero(counts)[0]
    loss = np.zeros(len(x))
    loss[rows] = lse[rows] - logits[rows, target[rows]]
    out = {"loss": loss, "lse": lse}
    if gl is None:
        return out
    g = np.exp(logits - lse[:, None])
    g[rows, target[rows]] -= 1.0
    scale = np.zeros(len(x))
    scale[rows] = gl[rows]
    g = np.where(counts[:, None], g * scale[:, None], 0.0)
    xz = np.where(counts[:, None], x, 0.0)
    out["grad_x"], out["grad_w"] = g @ w, g.T @ xz
    out["scale_grad_x"], out["scale_grad_w"] = np.abs(g) @ np.abs(w), np.abs(g).T @ np.abs(xz)
    return out
