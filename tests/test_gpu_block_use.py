"""The operators of delta-rule language models as they are used: together, with gradients,
in captured graphs, on other streams, and on arrays of more than 2^31 elements.

Bounds of the runs together.  The delta rule is off by 4e-5 of the usual size of its
output forward and 1.2e-4 backward; each passes a norm, a product and a softmax, which
keep relative errors to within a factor of two a way: 4 * 1.6e-4 = 6.4e-4 of the usual
size (the root mean square) of a tensor."""
import pytest
import torch

import linear_recurrence_scan_diagonal_amd as lrs
import block_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOGETHER = 6.4e-4


def f64(t):
    return t.detach().cpu().double()


def rms_close(name, got, ref, tol):
    off, size = (f64(got) - f64(ref)).abs().max(), f64(ref).square().mean().sqrt()
    assert off <= tol * size, (name, float(off / size))


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, gamma):
        y, s, rstd = lrs.rmsnorm_fwd(x, gamma, residual, save=True)
        ctx.save_for_backward(x if s is None else s, gamma, rstd)
        ctx.add = residual is not None
        return (y, s) if ctx.add else y

    @staticmethod
    def backward(ctx, gy, gs=None):
        s, gamma, rstd = ctx.saved_tensors
        gx, gg = lrs.rmsnorm_bwd(s, gamma, rstd, gy.contiguous(), None if gs is None else gs.contiguous())
        return gx, gx if ctx.add else None, gg


class Delta(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_decay, beta, reset):
        ck = lrs.gdr_checkpoints(k, v)
        ctx.save_for_backward(q, k, v, log_decay, beta, ck)
        ctx.reset = reset
        return lrs.gdr_fwd(q, k, v, log_decay, beta, reset=reset, checkpoints=ck)

    @staticmethod
    def backward(ctx, go):
        *inputs, ck = ctx.saved_tensors
        return (*lrs.gdr_bwd(*inputs, ck, go.contiguous(), reset=ctx.reset)[:5], None)


class LogProbs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, target):
        logprob, entropy, lse, _, _ = lrs.logprobs_fwd(logits, target)
        ctx.save_for_backward(logits, target, lse, entropy)
        return logprob, entropy

    @staticmethod
    def backward(ctx, gl, ge):
        return lrs.logprobs_bwd(*ctx.saved_tensors, gl.contiguous(), ge.contiguous()), None


def plain_norm(x, residual, gamma):
    s = x if residual is None else x + residual
    y = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + 1e-6) * gamma
    return y if residual is None else (y, s)


def plain_delta(q, k, v, log_decay, beta, reset):
    T, B, H, V = v.shape
    q, k = (x.repeat_interleave(H // x.shape[2], dim=2) for x in (q, k))
    S, o = v.new_zeros(B, H, k.shape[3], V), []
    for t in range(T):
        S = S * torch.exp(log_decay[t])[..., None, None] * (reset[t] == 0)[:, None, None, None]
        u = beta[t][..., None] * (v[t] - (S * k[t][..., None]).sum(2))
        S = S + k[t][..., None] * u[..., None, :]
        o.append(k.shape[3] ** -0.5 * (S * q[t][..., None]).sum(2))
    return torch.stack(o)


def plain_logprobs(logits, target):
    lp = logits - torch.logsumexp(logits, 1, keepdim=True)
    ok = target >= 0
    return torch.where(ok, lp.gather(1, target.clamp(min=0)[:, None])[:, 0], 0.0), -(lp.exp() * lp).sum(1)


H, HK, K, V, D, VOCAB = 4, 2, 24, 20, 48, 301


def weights():
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(table=n(VOCAB, D), gamma1=1 + 0.1 * n(D), w=n(D, 2 * HK * K + H * V + 2 * H) / D ** 0.5,
                out=n(H * V, D) / (H * V) ** 0.5, gamma2=1 + 0.1 * n(D), head=n(D, VOCAB) / D ** 0.5)


def parts(p, x, norm):
    """The inputs of the delta rule for x [..., D]."""
    lead = x.shape[:-1]
    z = norm(x, None, p["gamma1"]) @ p["w"]
    a, b, c, d = HK * K, 2 * HK * K, 2 * HK * K + H * V, 2 * HK * K + H * V + H
    unit = lambda r: r / r.square().sum(-1, keepdim=True).add(1e-6).sqrt()  # noqa: E731
    q, k = unit(z[..., :a].reshape(*lead, HK, K)), unit(z[..., a:b].reshape(*lead, HK, K))
    v = z[..., b:c].reshape(*lead, H, V).contiguous()
    return q, k, v, -torch.nn.functional.softplus(z[..., c:d]).contiguous(), torch.sigmoid(z[..., d:]).contiguous()


def tail(p, x, o, norm):
    y, _ = norm((o.flatten(-2) @ p["out"]).contiguous(), x, p["gamma2"])
    return y @ p["head"]


def steps(p, tokens, target, reset, norm, delta, logprobs, weight):
    x = p["table"][tokens]
    logits = tail(p, x, delta(*parts(p, x, norm), reset), norm)
    lp, ent = logprobs(logits.flatten(0, 1), target.flatten())
    return logits, -(weight * lp).sum() - 0.01 * ent.sum()


def batch(T=150, B=3):
    g = torch.Generator().manual_seed(2)
    tokens = torch.randint(0, VOCAB, (T, B), generator=g)
    target = torch.randint(0, VOCAB, (T, B), generator=g)
    target[T - 10:, 1] = -100
    reset = (torch.rand(T, B, generator=g) < 0.03).to(torch.uint8)
    return tokens, target, reset, torch.randn(T * B, generator=g)


def test_together():
    """Norm, delta rule, residual norm, head and weighted log probabilities with entropy."""
    tokens, target, reset, weight = batch()
    ours = {k: v.to(DEV).requires_grad_() for k, v in weights().items()}
    plain = {k: v.double().requires_grad_() for k, v in weights().items()}
    got, loss = steps(ours, tokens.to(DEV), target.to(DEV), reset.to(DEV), Norm.apply, Delta.apply, LogProbs.apply, weight.to(DEV))
    loss.backward()
    want, ref = steps(plain, tokens, target, reset, plain_norm, plain_delta, plain_logprobs, weight.double())
    ref.backward()
    rms_close("logits", got, want, TOGETHER)
    for k in ours:
        rms_close(k, ours[k].grad, plain[k].grad, TOGETHER)


def test_prompt_and_single_tokens():
    """A prompt, then one token at a time from its state: the logits and the alternatives'
    log probabilities of the whole sequence at once."""
    tokens, _, _, _ = batch(T=90)
    p = {k: v.to(DEV) for k, v in weights().items()}
    norm = lambda x, r, g: lrs.rmsnorm_fwd(x.contiguous(), g, r)[:2] if r is not None else lrs.rmsnorm_fwd(x, g)[0]  # noqa: E731
    x = p["table"][tokens.to(DEV)]
    whole = tail(p, x, lrs.gdr_fwd(*parts(p, x, norm)), norm)
    n = 71
    o, state = lrs.gdr_fwd(*parts(p, x[:n], norm), want_state=True)
    rms_close("prompt", tail(p, x[:n], o, norm), whole[:n], TOGETHER)
    for t in range(n, 90):
        xt = x[t].contiguous()
        logits = tail(p, xt, lrs.gdr_step(*parts(p, xt, norm), state), norm)
        rms_close(t, logits, whole[t], TOGETHER)
        some = torch.zeros(3, dtype=torch.int64, device=DEV)
        _, _, _, ids, lps = lrs.logprobs_fwd(logits, some, top=5)
        want = torch.log_softmax(f64(logits), 1)
        rms_close(t, lps, want.gather(1, ids.cpu()), 1e-5)


def test_delta_rule_gradient_against_differences():
    g = torch.Generator().manual_seed(4)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    T, B = 81, 2
    unit = lambda r: r / r.norm(dim=-1, keepdim=True)  # noqa: E731
    t = dict(q=unit(n(T, B, 2, 12)), k=unit(n(T, B, 2, 12)), v=n(T, B, 4, 9), log_decay=-torch.rand(T, B, 4, generator=g),
             beta=torch.sigmoid(n(T, B, 4)))
    state0, go, gs = n(B, 4, 12, 9), n(T, B, 4, 9), n(B, 4, 12, 9)
    reset = (torch.rand(T, B, generator=g) < 0.04).to(torch.uint8)
    dev = {k: v.to(DEV) for k, v in t.items()}
    ck = lrs.gdr_checkpoints(dev["k"], dev["v"])
    lrs.gdr_fwd(*dev.values(), reset=reset.to(DEV), state0=state0.to(DEV), checkpoints=ck)
    grads = lrs.gdr_bwd(*dev.values(), ck, go.to(DEV), reset=reset.to(DEV), grad_state=gs.to(DEV))
    x = {k: v.double() for k, v in (*t.items(), ("state0", state0))}
    for name, grad in zip(x, grads):
        d = n(*x[name].shape).double()

        def f(h):
            y = dict(x, **{name: x[name] + h * d})
            r = R.gdr(y["q"], y["k"], y["v"], y["log_decay"], y["beta"], 12 ** -0.5, reset, y["state0"])
            return (r["o"] * go.double()).sum() + (r["state"] * gs.double()).sum()
        slope = (f(1e-5) - f(-1e-5)) / 2e-5
        assert abs((f64(grad) * d).sum() - slope) <= 1.2e-4 * (f64(grad) * d).square().sum().sqrt(), name


def calls(dtype=torch.bfloat16, seed=0):
    """A pass through each operator over fixed inputs: {name: function of nothing}."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    T, B = 200, 2
    q, k, v = 0.2 * n(T, B, 2, 32), 0.2 * n(T, B, 2, 32), n(T, B, 4, 48)
    q, k, v, go = (t.to(dtype) for t in (q, k, v, n(T, B, 4, 48)))
    ld, beta = -torch.rand(T, B, 4, generator=g, device=DEV), torch.rand(T, B, 4, generator=g, device=DEV)
    reset = (torch.rand(T, B, generator=g, device=DEV) < 0.05).to(torch.uint8)
    x, r, gy, gamma = n(77, 640).to(dtype), n(77, 640).to(dtype), n(77, 640).to(dtype), n(640)
    logits, target = (4 * n(33, 9001)).to(dtype), torch.randint(0, 9001, (33,), generator=g, device=DEV)
    gl, ge = n(33), n(33)
    state = n(5, 4, 32, 48)
    slots = torch.tensor([3, 1], dtype=torch.int32, device=DEV)

    def delta():
        ck = lrs.gdr_checkpoints(k, v)
        o, s = lrs.gdr_fwd(q, k, v, ld, beta, reset=reset, want_state=True, checkpoints=ck)
        return (o, s, *lrs.gdr_bwd(q, k, v, ld, beta, ck, go, reset=reset))

    def step():
        s = state.clone()
        return lrs.gdr_step(q[0], k[0], v[0], ld[0], beta[0], s, slots), s

    def norm():
        y, s, rstd = lrs.rmsnorm_fwd(x, gamma, r, save=True)
        return (y, s, rstd, *lrs.rmsnorm_bwd(s, gamma, rstd, gy))

    def norm8():
        b, sc, s = lrs.rmsnorm_fwd_fp8(x, gamma, r)
        return b.view(torch.uint8), sc, s

    def probs():
        lp, h, lse, ids, tops = lrs.logprobs_fwd(logits, target, top=9)
        return lp, h, lse, ids, tops, lrs.logprobs_bwd(logits, target, lse, h, gl, ge)
    return dict(delta=delta, step=step, norm=norm, norm8=norm8, probs=probs)


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("name", ["delta", "step", "norm", "norm8", "probs"])
def test_captured(name):
    """Two graphs of different inputs, replayed in turn with eager calls between."""
    fs = [calls(seed=s)[name] for s in (0, 1)]
    want = [[t.clone() for t in f()] for f in fs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    side = torch.cuda.Stream()
    for f in fs:
        graph = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            f()
        torch.cuda.current_stream().wait_stream(side)
        with torch.cuda.graph(graph):
            outs.append(f())
        graphs.append(graph)
    for turn in range(4):
        for i in (0, 1) if turn % 2 else (1, 0):
            for t in outs[i]:
                t.zero_()
            graphs[i].replay()
            assert same(fs[1 - i](), want[1 - i]), turn
            torch.cuda.synchronize()
            assert same(outs[i], want[i]), turn
    for i in (0, 1):  # one behind the other, no wait between
        graphs[i].replay()
    torch.cuda.synchronize()
    assert same(outs[0], want[0]) and same(outs[1], want[1])


def test_gradients_captured_beside_an_eager_graph():
    """A training step captured, on leaves of its own that share the values, while an eager
    graph of the weights lives."""
    tokens, target, reset, weight = (t.to(DEV) for t in batch(T=70, B=2))
    p = {k: v.to(DEV).requires_grad_() for k, v in weights().items()}
    args = (tokens, target, reset, Norm.apply, Delta.apply, LogProbs.apply, weight)
    _, alive = steps(p, *args)
    want = torch.autograd.grad(steps(p, *args)[1], list(p.values()))
    mine = {k: v.detach().requires_grad_() for k, v in p.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(steps(mine, *args)[1], list(mine.values()))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(steps(mine, *args)[1], list(mine.values()))
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for name, a, b in zip(p, got, want):
            if name != "table":  # torch adds its rows up in any order
                rms_close(name, a, b, 1e-5)
    alive.backward()


@pytest.mark.parametrize("name", ["delta", "step", "norm", "norm8", "probs"])
def test_two_streams(name):
    fs = [calls(seed=s)[name] for s in (0, 1)]
    want = [[t.clone() for t in f()] for f in fs]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in fs], [[], []]
    for _ in range(5):
        for i, f in enumerate(fs):
            with torch.cuda.stream(streams[i]):
                outs[i].append(f())
    torch.cuda.synchronize()
    assert all(same(o, want[i]) for i in (0, 1) for o in outs[i])


def test_norm_of_more_than_2_31_elements():
    R_, D_, n = 1_050_003, 2051, 64
    x = torch.randn(R_, D_, device=DEV, dtype=torch.bfloat16)
    gamma = torch.randn(D_, device=DEV)
    gy = torch.zeros_like(x)
    gy[-n:] = torch.randn(n, D_, device=DEV).bfloat16()
    y, _, rstd = lrs.rmsnorm_fwd(x, gamma, save=True)
    gx, gg = lrs.rmsnorm_bwd(x, gamma, rstd, gy)
    y1, _, rstd1 = lrs.rmsnorm_fwd(x[-n:].contiguous(), gamma, save=True)
    gx1, gg1 = lrs.rmsnorm_bwd(x[-n:].contiguous(), gamma, rstd1, gy[-n:].contiguous())
    assert gx[: R_ - n].abs().max() == 0
    for name, a, b in (("y", y[-n:], y1), ("rstd", rstd[-n:], rstd1), ("grad_x", gx[-n:], gx1), ("grad_gamma", gg, gg1)):
        tol = 2.0 ** -7 if a.dtype == torch.bfloat16 else 1e-5
        assert ((f64(a) - f64(b)).abs() <= tol * f64(b).abs() + 1e-5 * f64(b).square().mean().sqrt()).all(), name
    del y, gx, gy
    q, scales, _ = lrs.rmsnorm_fwd_fp8(x, gamma)
    q1, scales1, _ = lrs.rmsnorm_fwd_fp8(x[-n:].contiguous(), gamma)
    assert torch.allclose(scales[-n:], scales1, rtol=1e-6, atol=0)
    # a scale's last bit may move a value across a border between two bytes, a step of 2^-3
    a, b = f64(q[-n:].float()), f64(q1.float())
    assert ((a - b).abs() <= 2.0 ** -3 * b.abs() + 2.0 ** -9).all() and (a != b).double().mean() < 1e-3


def test_log_probabilities_of_more_than_2_31_elements():
    N, V_, n = 66_001, 32_771, 600
    logits = torch.randn(N, V_, device=DEV, dtype=torch.bfloat16)
    target = torch.randint(0, V_, (N,), device=DEV)
    gl, ge = torch.randn(N, device=DEV), torch.randn(N, device=DEV)
    got = lrs.logprobs_fwd(logits, target, top=4)
    last = logits[-n:].contiguous()
    want = lrs.logprobs_fwd(last, target[-n:], top=4)
    assert torch.equal(got[3][-n:], want[3])
    for i in (0, 1, 2, 4):
        assert torch.allclose(got[i][-n:], want[i], rtol=2e-6, atol=2e-6)
    g1 = lrs.logprobs_bwd(last, target[-n:], want[2], want[1], gl[-n:], ge[-n:])
    g = lrs.logprobs_bwd(logits, target, got[2], got[1], gl, ge, out=logits)
    assert ((g[-n:].float() - g1.float()).abs() <= 2.0 ** -7 * g1.float().abs() + 1e-9).all()


def test_delta_rule_of_more_than_2_31_elements():
    T, B, n = 64 * 2049, 8, 192
    q, k = (torch.randn(T, B, 8, 128, device=DEV, dtype=torch.bfloat16).mul_(128 ** -0.5) for _ in range(2))
    v, go = (torch.randn(T, B, 16, 128, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    ld, beta = -torch.rand(T, B, 16, device=DEV), torch.rand(T, B, 16, device=DEV)
    reset = torch.zeros(T, B, device=DEV, dtype=torch.uint8)
    reset[T - n] = 1
    ck = lrs.gdr_checkpoints(k, v)
    o, state = lrs.gdr_fwd(q, k, v, ld, beta, reset=reset, want_state=True, checkpoints=ck)
    got = (o, state, *lrs.gdr_bwd(q, k, v, ld, beta, ck, go, reset=reset)[:5])
    assert not bool(torch.isnan(o[:: 64 * 128]).any())
    q, k, v, go, ld, beta = (t[-n:].contiguous() for t in (q, k, v, go, ld, beta))
    ck = lrs.gdr_checkpoints(k, v)
    o, state = lrs.gdr_fwd(q, k, v, ld, beta, want_state=True, checkpoints=ck)
    want = (o, state, *lrs.gdr_bwd(q, k, v, ld, beta, ck, go)[:5])
    for i, (a, b) in enumerate(zip(got, want)):
        a, b = f64(a if i == 1 else a[-n:]), f64(b)
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 1.2e-4 * b.square().mean().sqrt()).all(), i
