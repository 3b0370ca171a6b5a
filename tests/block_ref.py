"""Plain fp64 forms of the operators of delta-rule language models
(include/lrs_block.h): one time step or one row after the other, on the CPU, sharing no
code with the device path."""
import torch


def gdr(q, k, v, log_decay, beta, scale, reset=None, state0=None, grad_o=None, grad_state=None):
    """Forward, and with grad_o the gradients, of the gated delta rule on float64
    arrays: q, k [T,B,Hk,K], v [T,B,H,V], gates [T,B,H]."""
    T, B, H, V = v.shape
    Hk, K = k.shape[2:]
    share = H // Hk
    q, k = (x.repeat_interleave(share, dim=2) for x in (q, k))
    cut = torch.zeros(T, B, dtype=torch.bool) if reset is None else reset != 0
    S = torch.zeros(B, H, K, V, dtype=torch.float64) if state0 is None else state0
    a = torch.exp(log_decay)
    o, kept, miss, u = torch.zeros_like(v), [], torch.zeros_like(v), torch.zeros_like(v)
    for t in range(T):
        # a restart drops the state, whatever it holds
        S = torch.where(cut[t][:, None, None, None], 0.0, S * a[t][..., None, None])
        kept.append(S)
        miss[t] = v[t] - torch.einsum("bhkv,bhk->bhv", S, k[t])
        u[t] = beta[t][..., None] * miss[t]
        S = S + k[t][..., None] * u[t][..., None, :]
        o[t] = scale * torch.einsum("bhkv,bhk->bhv", S, q[t])
    out = {"o": o, "state": S}
    if grad_o is None:
        return out
    gS = torch.zeros_like(S) if grad_state is None else grad_state
    gq, gk, gv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    gg, gb = torch.zeros_like(beta), torch.zeros_like(beta)
    for t in range(T - 1, -1, -1):
        go = scale * grad_o[t]
        gq[t] = torch.einsum("bhkv,bhv->bhk", kept[t] + k[t][..., None] * u[t][..., None, :], go)
        gS = gS + q[t][..., None] * go[..., None, :]
        gu = torch.einsum("bhkv,bhk->bhv", gS, k[t])
        gv[t] = beta[t][..., None] * gu
        gb[t] = (gu * miss[t]).sum(-1)
        gk[t] = (torch.einsum("bhkv,bhv->bhk", gS, u[t]) -
                 torch.einsum("bhkv,bhv->bhk", kept[t], gv[t]))
        gS = gS - k[t][..., None] * gv[t][..., None, :]
        c = cut[t][:, None]
        gg[t] = torch.where(c, 0.0, (gS * kept[t]).sum((-1, -2)))
        gS = torch.where(c[..., None, None], 0.0, gS * a[t][..., None, None])
    gq, gk = (x.unflatten(2, (Hk, share)).sum(3) for x in (gq, gk))
    out.update(grad_q=gq, grad_k=gk, grad_v=gv, grad_log_decay=gg, grad_beta=gb, grad_state0=gS)
    return out


def rmsnorm(s, gamma, eps, gy=None, gsum=None):
    rstd = 1.0 / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    xh = s * rstd
    out = {"y": xh * gamma, "rstd": rstd[:, 0]}
    if gy is None:
        return out
    g = gy * gamma
    dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
    out["grad_x"] = dx if gsum is None else dx + gsum
    out["grad_gamma"] = (gy * xh).sum(0)
    out["scale_grad_gamma"] = (gy * xh).abs().sum(0)
    return out


def e4m3_grid():
    """The values of e4m3 (finite, not negative), ascending."""
    return torch.tensor(sorted({m * 2.0 ** -9 for m in range(8)} |
                               {(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)
                                if (e, m) != (15, 7)}), dtype=torch.float64)


def logprobs(logits, target, gl=None, ge=None):
    """logits [N,V] float64 (finite or -inf, not a whole row of it)."""
    N, V = logits.shape
    m = logits.max(1).values
    e = torch.exp(logits - m[:, None])
    lse = m + torch.log(e.sum(1))
    lp = logits - lse[:, None]
    p = torch.exp(lp)
    plp = torch.where(p > 0, p * lp, 0.0)
    entropy = -plp.sum(1)
    ok = (target >= 0) & (target < V)
    rows = torch.nonzero(ok)[:, 0]
    logprob = torch.zeros(N, dtype=torch.float64)
    logprob[rows] = lp[rows, target[rows]]
    out = {"logprob": logprob, "entropy": entropy, "lse": lse, "lp": lp}
    if gl is None:
        return out
    w = torch.where(ok, gl, 0.0)
    g = -p * w[:, None]
    g[rows, target[rows]] += w[rows]
    if ge is not None:
        g = g - ge[:, None] * (plp + p * entropy[:, None])
    out["grad_logits"] = g
    return out


def tops(logits, top):
    """Indices of the largest, the lower index first where they are equal (-0 and 0 are),
    NaN above all; [N,top]."""
    x = torch.where(torch.isnan(logits), torch.inf, logits.clamp(max=torch.finfo(torch.float64).max))
    return torch.sort(-x, dim=1, stable=True).indices[:, :top]
