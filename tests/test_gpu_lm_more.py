"""The language-model operators in captured graphs, on another stream, on arrays of
more than 2^31 elements, against differences of their own forward, and with values
that are not finite."""
import pytest
import torch

import linear_recurrence_scan_diagonal_amd as lrs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rand(*shape, seed=0, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def glr_params(D, seed=1):
    return dict(bias_r=0.3 * rand(D, seed=seed), bias_i=0.3 * rand(D, seed=seed + 1),
                decay=rand(D, seed=seed + 2) - 4.0)


def glr_train_step(T, B, D, dtype):
    z, gh, h0 = rand(T, B, 3 * D, dtype=dtype), rand(T, B, D, seed=3, dtype=dtype), rand(B, D, seed=4)
    p, reset = glr_params(D), rand(T, B, seed=5) > 2.0

    def step():
        parts = z.chunk(3, dim=-1)
        ck = lrs.glr_checkpoints(parts[0])
        h, last = lrs.glr_fwd(*parts, **p, reset=reset, h0=h0, want_h_last=True, checkpoints=ck)
        return (h, last) + lrs.glr_bwd(*parts, **p, checkpoints=ck, grad_h=gh, reset=reset)
    return step


def norm_train_step(R, D, dtype):
    x, r, gy = (rand(R, D, seed=s, dtype=dtype) for s in (0, 1, 2))
    gamma, beta = 1 + 0.1 * rand(D, seed=3), rand(D, seed=4)

    def step():
        y, s, mean, rstd = lrs.layernorm_fwd(x, gamma, beta, residual=r, save=True)
        return (y, s, mean, rstd) + lrs.layernorm_bwd(s, gamma, mean, rstd, gy, grad_sum=gy)
    return step


def loss_step(N, V, D, dtype):
    x, w = rand(N, D, dtype=dtype), rand(V, D, seed=1, dtype=dtype)
    target = torch.arange(N, device=DEV) * 7 % (V + 1)  # V: ignored
    gl = rand(N, seed=2)

    def step():
        return lrs.linear_ce_fwd(x, w, target) + lrs.linear_ce_fwd_bwd(x, w, target, gl)
    return step


def decode_step(B, D, dtype):
    z, p, pool = rand(B, 3 * D, dtype=dtype), glr_params(D), rand(2 * B, D, seed=3)
    slots = (torch.arange(B, device=DEV) * 2 % (2 * B + 1)).int()
    start = pool.clone()

    def step():
        pool.copy_(start)
        return (lrs.glr_step(*z.chunk(3, dim=-1), **p, state=pool, slots=slots), pool)
    return step


STEPS = {
    "glr few channels": lambda: glr_train_step(700, 2, 96, torch.bfloat16),
    "glr many channels": lambda: glr_train_step(130, 70, 512, torch.bfloat16),
    "glr fp32": lambda: glr_train_step(300, 3, 77, torch.float32),
    "norm": lambda: norm_train_step(1500, 640, torch.bfloat16),
    "norm wide": lambda: norm_train_step(300, 9001, torch.float32),
    "loss bf16": lambda: loss_step(300, 5000, 96, torch.bfloat16),
    "loss odd": lambda: loss_step(123, 777, 65, torch.bfloat16),
    "loss fp32": lambda: loss_step(300, 1000, 96, torch.float32),
    "decode": lambda: decode_step(9, 200, torch.bfloat16),
}


@pytest.mark.parametrize("name", STEPS)
def test_graph_replay(name):
    """Every replay gives the eager call's bits, with unrelated eager work between."""
    step = STEPS[name]()
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    other = norm_train_step(77, 130, torch.float32)
    for rep in range(4):
        for t in got:
            t.fill_(1e30)
        other()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (g, w) in enumerate(zip(got, want)):
            assert torch.equal(g, w), (rep, i)


@pytest.mark.parametrize("name", STEPS)
def test_other_stream(name):
    """The work goes to the current stream: it follows what that stream did before."""
    step = STEPS[name]()
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        got = step()
        copies = [t.clone() for t in got]
    stream.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(copies, want))


def test_norm_past_32_bit_offsets():
    """Rows do not depend on each other: the last ones have the bits of a small call."""
    R, D = 2_200_000, 1024
    x = torch.empty(R, D, dtype=torch.bfloat16, device=DEV).normal_()
    gamma, beta = 1 + 0.1 * rand(D), rand(D, seed=1)
    y, s, mean, rstd = lrs.layernorm_fwd(x, gamma, beta, residual=x, save=True)
    gx, gg, gb = lrs.layernorm_bwd(s, gamma, mean, rstd, y)
    tail = slice(R - 70, R)
    ty, ts, tm, tr = lrs.layernorm_fwd(x[tail], gamma, beta, residual=x[tail], save=True)
    tgx, _, _ = lrs.layernorm_bwd(ts, gamma, tm, tr, ty)
    for a, b in ((y[tail], ty), (s[tail], ts), (mean[tail], tm), (rstd[tail], tr), (gx[tail], tgx)):
        assert torch.equal(a, b)
    # the sums over rows, in pieces; 4000 rounded products of size 1 a piece and column
    want = torch.zeros(D, dtype=torch.float64, device=DEV)
    for i in range(0, R, 200_000):
        want += y[i:i + 200_000].double().sum(0)
    assert ((gb.double() - want).abs() <= 1e-5 * (1 + R)).all()


def test_glr_past_32_bit_offsets():
    """The last steps are those of a call that goes on from the state before them."""
    T, B, D = 70_000, 8, 4096
    cut = T - 500
    z = torch.empty(T, B, 3 * D, dtype=torch.bfloat16, device=DEV).normal_()
    p = glr_params(D)
    parts = z.chunk(3, dim=-1)
    ck = lrs.glr_checkpoints(parts[0])
    h, last = lrs.glr_fwd(*parts, **p, want_h_last=True, checkpoints=ck)
    _, mid = lrs.glr_fwd(*(v[:cut] for v in parts), **p, want_h_last=True)
    tail = [v[cut:] for v in parts]
    tck = lrs.glr_checkpoints(tail[0])
    th, tlast = lrs.glr_fwd(*tail, **p, h0=mid, want_h_last=True, checkpoints=tck)
    assert ((last - tlast).abs() <= 1e-5 * (1 + tlast.abs())).all()
    bf = 2.0 ** -7 + 1e-5  # one unit in the last place where a rounding falls the other way
    assert ((h[cut:].float() - th.float()).abs() <= bf * (1 + th.float().abs())).all()
    grad_z = torch.empty_like(z)
    lrs.glr_bwd(*parts, **p, checkpoints=ck, grad_h=h, grad_z=grad_z.chunk(3, dim=-1))
    want = lrs.glr_bwd(*tail, **p, checkpoints=tck, grad_h=th)
    # the gradients follow grad_h, whose own roundings may differ by a unit and are
    # summed over the memory: 2^-7 of the largest value
    for g, w in zip(grad_z[cut:].chunk(3, dim=-1), want[:3]):
        assert (g.float() - w.float()).abs().max() <= 2.0 ** -7 * w.float().abs().max()


def test_loss_past_32_bit_offsets():
    N, V, D = 1 << 20, 64, 2304
    x = torch.empty(N, D, dtype=torch.bfloat16, device=DEV).normal_()
    w = (0.05 * rand(V, D)).bfloat16()
    target = torch.arange(N, device=DEV) % V
    gl = torch.full((N,), 1.0, device=DEV)
    loss, lse, gx, gw = lrs.linear_ce_fwd_bwd(x, w, target, gl)
    tail = slice(N - 300, N)
    tl, tlse, tgx, _ = lrs.linear_ce_fwd_bwd(x[tail], w, target[tail], gl[tail])
    assert ((loss[tail] - tl).abs() <= 1e-5 * (1 + tl.abs())).all()
    assert ((lse[tail] - tlse).abs() <= 1e-5 * (1 + tlse.abs())).all()
    assert (gx[tail].float() - tgx.float()).abs().max() <= 2.0 ** -7 * tgx.float().abs().max()
    # every part of the sum over rows, from calls on an eighth of them
    want = sum(lrs.linear_ce_fwd_bwd(x[i:i + N // 8], w, target[i:i + N // 8], gl[i:i + N // 8])[3]
               .double() for i in range(0, N, N // 8))
    # eight roundings of 2^-9 of a part, and one of the whole
    assert (gw.double() - want).abs().max() <= 2.0 ** -6 * want.abs().max()


def difference(f, t, direction, eps):
    """Central difference of f along a direction of t."""
    keep = t.clone()
    t.copy_(keep + eps * direction)
    hi = f()
    t.copy_(keep - eps * direction)
    lo = f()
    t.copy_(keep)
    return (hi - lo) / (2 * eps)


# Differences in fp32: f is a sum of n products of size 1, known to about 1e-6 sqrt(n)
# (each value to 1e-6), so a difference over 2 eps = 0.02 is known to 1e-4 sqrt(n); the
# third derivative adds eps^2 = 1e-4 of a few times the value.  sqrt(n) is about 50
# here, the derivative along a unit normal direction about as large: 2 % of 1 + sqrt(n).

def test_glr_differences():
    T, B, D = 70, 2, 20
    parts = [rand(T, B, D, seed=s) for s in (0, 1, 2)]
    p, h0, gh = glr_params(D), rand(B, D, seed=6), rand(T, B, D, seed=7)
    p["decay"] += 2.0
    reset = rand(T, B, seed=8) > 1.8

    def f():
        return float((lrs.glr_fwd(*parts, **p, reset=reset, h0=h0).double() * gh.double()).sum())
    ck = lrs.glr_checkpoints(parts[0])
    lrs.glr_fwd(*parts, **p, reset=reset, h0=h0, checkpoints=ck)
    grads = lrs.glr_bwd(*parts, **p, checkpoints=ck, grad_h=gh, reset=reset)
    bound = 0.02 * (1 + (T * B * D) ** 0.5)
    for i, (t, g) in enumerate(zip([*parts, p["bias_r"], p["bias_i"], p["decay"], h0], grads)):
        d = rand(*t.shape, seed=20 + i)
        want = difference(f, t, d, 0.01)
        assert abs(float((g.double() * d.double()).sum()) - want) <= bound, i


def test_norm_differences():
    R, D = 40, 60
    x, r, gy, gs = (rand(R, D, seed=s) for s in range(4))
    gamma, beta = 1 + 0.1 * rand(D, seed=4), rand(D, seed=5)

    def f():
        y, s, _, _ = lrs.layernorm_fwd(x, gamma, beta, residual=r)
        return float((y.double() * gy + s.double() * gs).sum())
    _, s, mean, rstd = lrs.layernorm_fwd(x, gamma, beta, residual=r, save=True)
    gx, gg, gb = lrs.layernorm_bwd(s, gamma, mean, rstd, gy, grad_sum=gs)
    bound = 0.02 * (1 + (R * D) ** 0.5)
    for i, (t, g) in enumerate(((x, gx), (r, gx), (gamma, gg), (beta, gb))):
        d = rand(*t.shape, seed=20 + i)
        assert abs(float((g.double() * d.double()).sum()) - difference(f, t, d, 0.01)) <= bound, i


def test_loss_differences():
    N, V, D = 60, 90, 30
    x, w, gl = rand(N, D), 0.3 * rand(V, D, seed=1), rand(N, seed=2)
    target = torch.arange(N, device=DEV) * 5 % (V + 3)

    def f():
        return float((lrs.linear_ce_fwd(x, w, target)[0].double() * gl).sum())
    _, _, gx, gw = lrs.linear_ce_fwd_bwd(x, w, target, gl)
    bound = 0.02 * (1 + (N * D) ** 0.5)
    for i, (t, g) in enumerate(((x, gx), (w, gw))):
        d = rand(*t.shape, seed=20 + i)
        assert abs(float((g.double() * d.double()).sum()) - difference(f, t, d, 0.01)) <= bound, i


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("others", [0.0, 1.0])
def test_nan_gradient_of_a_loss(dtype, others):
    """It reaches its row's grad_x and all of grad_w, and no other row of grad_x, also
    where every other row's gradient is 0."""
    N, V, D = 50, 130, 40
    x, w = rand(N, D, dtype=dtype), rand(V, D, seed=1, dtype=dtype)
    target = torch.arange(N, device=DEV)
    gl = torch.full((N,), others, device=DEV)
    gl[7] = float("nan")
    _, _, gx, gw = lrs.linear_ce_fwd_bwd(x, w, target, gl)
    rows = torch.arange(N, device=DEV) != 7
    assert torch.isnan(gx[7]).all() and torch.isnan(gw).all()
    assert torch.isfinite(gx[rows]).all()
    assert bool((gx[rows] == 0).all()) == (others == 0.0)


def test_rows_without_a_gradient_may_overflow():
    """A row that counts, with a gradient of 0 and logits that are not finite, changes
    no other row's gradient."""
    N, V, D = 50, 130, 64
    x, w = rand(N, D, dtype=torch.bfloat16), rand(V, D, seed=1, dtype=torch.bfloat16)
    target, gl = torch.arange(N, device=DEV), torch.full((N,), 0.5, device=DEV)
    gl[11] = 0.0
    want = lrs.linear_ce_fwd_bwd(x, w, target, gl)
    x[11, 3] = float("inf")
    got = lrs.linear_ce_fwd_bwd(x, w, target, gl)
    assert torch.equal(got[2], want[2]) and torch.equal(got[3], want[3])


def test_classes_of_minus_infinity():
    """Logits of -inf (x > 0 where w is -inf) are classes of probability 0."""
    N, V, D = 33, 300, 16
    x = rand(N, D).abs().bfloat16()
    w = rand(V, D, seed=1).bfloat16()
    target = torch.full((N,), 299, device=DEV)
    w2 = torch.cat([w, w[:200].clone()])
    w2[300:, 0] = -float("inf")
    loss, lse = lrs.linear_ce_fwd(x, w2, target)
    want = torch.logsumexp(x.double() @ w.double().t(), 1)
    assert ((lse.double() - want).abs() <= 1e-5 * (1 + want.abs())).all()
    assert torch.isfinite(loss).all()


def test_many_short_rows():
    """Five million rows of 16 features: more than 2^32 / 1024."""
    R, D = 5_000_000, 16
    x, gamma, beta = rand(R, D, dtype=torch.bfloat16), 1 + 0.1 * rand(D, seed=1), rand(D, seed=2)
    y, _, mean, rstd = lrs.layernorm_fwd(x, gamma, beta, save=True)
    gx, _, _ = lrs.layernorm_bwd(x, gamma, mean, rstd, y)
    part = slice(R - 1000, R)
    ty, _, tm, tr = lrs.layernorm_fwd(x[part], gamma, beta, save=True)
    tgx, _, _ = lrs.layernorm_bwd(x[part], gamma, tm, tr, ty)
    assert torch.equal(y[part], ty) and torch.equal(gx[part], tgx)
