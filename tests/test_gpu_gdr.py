"""The gated delta rule on the GPU against the plain fp64 form.

Bounds.  A factor of a product is known to 2^-22, so a sum of products to 2^-21 of the
sum of its absolute terms; five products follow each other on the way to an output, and
the absolute terms of some 192 of random sign add up to 14 times their sum's usual size:
5 * 14 * 2^-21 = 3.4e-5 of the usual size of an output, 4e-5 here.  A gradient has up to
three such ways on top of each other: 1.2e-4.  The usual size is the root mean square of
what the reference gives for the sequence and head.  bf16 outputs are off by half a unit
in the last place more, 2^-8."""
import math

import pytest
import torch

import linear_recurrence_scan_diagonal_amd as lrs
import block_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
FWD, BWD = 4e-5, 1.2e-4


def make(T, B, H, Hk, K, V, dtype=torch.float32, seed=0, resets=0.0, decay=1.0, state=True):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    qk = n(T, B, 2 * Hk, K)
    qk = qk / qk.norm(dim=-1, keepdim=True)
    t = dict(q=qk[:, :, :Hk].to(dtype), k=qk[:, :, Hk:].to(dtype), v=n(T, B, H, V).to(dtype),
             log_decay=-decay * torch.rand(T, B, H, generator=g) ** 3,
             beta=torch.sigmoid(n(T, B, H)), grad_o=n(T, B, H, V).to(dtype))
    t["reset"] = (torch.rand(T, B, generator=g) < resets).to(torch.uint8) if resets else None
    t["state0"] = 0.3 * n(B, H, K, V) if state else None
    t["grad_state"] = 0.1 * n(B, H, K, V) if state else None
    return {k: None if v is None else v.contiguous().to(DEV) for k, v in t.items()}


def f64(t):
    return None if t is None else t.detach().cpu().double() if t.is_floating_point() else t.cpu()


def run(t, scale=None, train=True, grad_qkv=None):
    inputs = [t[n] for n in ("q", "k", "v", "log_decay", "beta")]
    ck = lrs.gdr_checkpoints(t["k"], t["v"]) if train else None
    o, state = lrs.gdr_fwd(*inputs, scale=scale, reset=t["reset"], state0=t["state0"], want_state=True,
                           checkpoints=ck)
    out = {"o": o, "state": state}
    if train:
        grads = lrs.gdr_bwd(*inputs, ck, t["grad_o"], scale=scale, reset=t["reset"],
                            grad_state=t["grad_state"], grad_qkv=grad_qkv)
        out.update(zip(("grad_q", "grad_k", "grad_v", "grad_log_decay", "grad_beta", "grad_state0"), grads))
    torch.cuda.synchronize()
    return out


def reference(t, scale=None):
    r = {k: f64(v) for k, v in t.items()}
    return R.gdr(r["q"], r["k"], r["v"], r["log_decay"], r["beta"],
                 r["k"].shape[-1] ** -0.5 if scale is None else scale, r["reset"], r["state0"],
                 r["grad_o"], r["grad_state"])


def usual(name, ref):
    """Root mean square a sequence and head, broadcast over the rest."""
    if name in ("state", "grad_state0"):
        return ref.square().mean((-1, -2), keepdim=True).sqrt()
    if name in ("grad_log_decay", "grad_beta"):
        return ref.square().mean(0, keepdim=True).sqrt()
    return ref.square().mean((0, -1), keepdim=True).sqrt()


def close(got, ref, factor=1.0):
    for name, x in got.items():
        y = ref[name]
        assert x.shape == y.shape
        tol = factor * (BWD if name.startswith("grad") else FWD)
        off = (f64(x) - y).abs()
        bound = tol * (usual(name, y) + y.abs())
        if x.dtype == torch.bfloat16:
            bound = bound + 2.0 ** -8 * y.abs()
        bad = off > bound + 1e-30
        assert not bad.any(), (name, float((off / (bound + 1e-30)).max()), torch.nonzero(bad)[:3].tolist())


SHAPES = [  # T, B, H, Hk, K, V
    (1, 1, 1, 1, 1, 1), (1, 3, 2, 1, 16, 16), (2, 1, 1, 1, 8, 5), (17, 2, 3, 3, 33, 7), (63, 1, 2, 2, 64, 64),
    (64, 2, 1, 1, 64, 128), (65, 1, 2, 1, 128, 64), (128, 1, 2, 2, 128, 128), (130, 3, 4, 2, 80, 72),
    (200, 2, 6, 2, 65, 33), (300, 1, 2, 2, 128, 160), (257, 2, 3, 1, 20, 200), (1000, 1, 1, 1, 100, 24)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES)
def test_parity(shape, dtype):
    t = make(*shape, dtype=dtype, seed=sum(shape))
    close(run(t), reference(t))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("resets", [0.004, 0.05, 0.5, 1.0])
def test_restarts(resets, dtype):
    t = make(200, 3, 4, 2, 40, 24, dtype=dtype, seed=5, resets=resets)
    close(run(t), reference(t))


@pytest.mark.parametrize("at", [[0], [63], [64], [65], [0, 64, 128], [1, 2, 3, 62, 63, 127, 191], [199]])
def test_restarts_at_chunk_borders(at):
    t = make(200, 2, 2, 1, 32, 40, seed=6)
    t["reset"] = torch.zeros(200, 2, dtype=torch.bool, device=DEV)
    t["reset"][at, 0] = True
    got, ref = run(t), reference(t)
    close(got, ref)
    assert (got["grad_log_decay"][at, 0] == 0).all()


def test_no_states():
    t = make(150, 2, 2, 2, 48, 48, state=False, seed=7)
    close(run(t), reference(t))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_slices_of_one_projection(dtype):
    """q, k and v as views of one array, gradients into views of another: the same bits as
    with arrays of their own."""
    T, B, H, Hk, K, V = 131, 2, 4, 2, 24, 40
    t = make(T, B, H, Hk, K, V, dtype=dtype, seed=8, resets=0.02)
    want = run(t)
    n, m = Hk * K, H * V
    pad = 3  # an odd row pitch
    z = torch.full((T, B, 2 * n + m + pad), 7.0, dtype=dtype, device=DEV)
    gz = torch.full_like(z, 7.0)

    def parts(x):
        return (x[..., :n].unflatten(-1, (Hk, K)), x[..., n:2 * n].unflatten(-1, (Hk, K)),
                x[..., 2 * n:2 * n + m].unflatten(-1, (H, V)))
    for view, name in zip(parts(z), "qkv"):
        view.copy_(t[name])
        t[name] = view
    got = run(t, grad_qkv=parts(gz))
    for name in want:
        assert torch.equal(got[name], want[name]), name
    assert (gz[..., 2 * n + m:] == 7.0).all()


def test_strong_and_absent_decay():
    t = make(200, 2, 2, 2, 32, 32, seed=9)
    t["log_decay"][:, :, 0] = 0.0
    t["log_decay"][::7, :, 1] = -80.0
    close(run(t), reference(t))
    # exp(-inf) = 0 drops the state as exp(-1e5) does, gradients included
    t["log_decay"][::7, :, 1] = -math.inf
    a = run(t)
    t["log_decay"][::7, :, 1] = -1e5
    b = run(t)
    for name in a:
        assert torch.equal(a[name], b[name]) and torch.isfinite(a[name]).all(), name
    close(b, reference(t))


def test_gates_at_their_ends():
    """beta 0 (nothing is written) and 1 or 2, and k of length 0."""
    t = make(200, 2, 3, 3, 32, 32, seed=10)
    t["beta"][:, :, 0] = 0.0
    t["beta"][:, :, 1] = 1.0
    t["beta"][::3, :, 2] = 2.0
    t["k"][::5] = 0.0
    close(run(t), reference(t))


@pytest.mark.parametrize("size", [1e-12, 1e8])
def test_range(size):
    """Powers of ten do not reach fp16: every row is scaled."""
    t = make(150, 1, 2, 1, 64, 48, seed=11, state=False)
    t["v"] *= size
    t["q"] *= size
    t["grad_o"] *= size
    got, ref = run(t), reference(t)
    close(got, ref)


def test_rows_of_different_size():
    """A document of small values behind one of large values in the same chunk keeps its digits."""
    t = make(64, 1, 1, 1, 32, 32, seed=12, state=False)
    t["reset"] = torch.zeros(64, 1, dtype=torch.uint8, device=DEV)
    t["reset"][32] = 1
    for n in ("v", "q", "grad_o"):
        t[n][:32] *= 1e10
    got, ref = run(t, train=True), reference(t)
    for name in ("o", "grad_v", "grad_q", "grad_k"):
        x, y = got[name][32:], ref[name][32:]
        assert ((f64(x) - y).abs() <= BWD * (y.square().mean().sqrt() + y.abs())).all(), name
    for name in ("grad_beta", "grad_log_decay"):
        x, y = got[name][32:], ref[name][32:]
        assert ((f64(x) - y).abs() <= BWD * (y.square().mean().sqrt() + y.abs())).all(), name


@pytest.mark.parametrize("what", ["q", "k", "v", "log_decay", "beta", "grad_o", "state0"])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_not_finite_stays_in_its_document(what, value):
    """A value that is not finite in one document, head and sequence changes nothing of
    the others, bit for bit."""
    T, B, H = 150, 2, 2
    t = make(T, B, H, 2, 24, 24, seed=13)
    t["reset"] = torch.zeros(T, B, dtype=torch.uint8, device=DEV)
    t["reset"][[20, 40, 64, 100], 0] = 1
    want = run(t)
    u = {k: None if v is None else v.clone() for k, v in t.items()}
    if what == "state0":
        u["state0"][0, 0, 3, 5] = value
        hit = range(0, 20)
    elif what in ("log_decay", "beta"):
        u[what][25, 0, 0] = value
        hit = range(20, 40)
    else:
        u[what][25, 0, 0, 3] = value
        hit = range(20, 40)
    got = run(u)
    keep = [i for i in range(T) if i not in hit]
    for name in want:
        x, y = got[name], want[name]
        if name in ("state", "grad_state0"):
            assert torch.equal(x[1], y[1]) and torch.equal(x[:, 1], y[:, 1]), name
            if name == "state" or what not in ("state0",):
                assert torch.equal(x[0, 0], y[0, 0]), name
        else:
            assert torch.equal(x[:, 1], y[:, 1]) and torch.equal(x[:, :, 1], y[:, :, 1]), name
            assert torch.equal(x[keep], y[keep]), name
    if what not in ("grad_o",):
        assert not torch.isfinite(got["o"][list(hit), 0, 0]).all()


def test_in_place_states():
    t = make(130, 2, 2, 2, 32, 48, seed=14)
    want = run(t)
    lib_state = t["state0"].clone()
    import ctypes
    from linear_recurrence_scan_diagonal_amd import block
    lib = block.load()
    T, B, H, Hk, K, V = 130, 2, 2, 2, 32, 48
    n = lib.lrs_gdr_workspace_bytes(T, B, H, Hk, K, V, 0)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    o = torch.empty_like(t["v"])
    p = lambda x: ctypes.c_void_p(x.data_ptr())  # noqa: E731
    rc = lib.lrs_gdr_fwd(p(t["q"]), Hk * K, p(t["k"]), Hk * K, p(t["v"]), H * V, p(t["log_decay"]),
                         p(t["beta"]), None, p(lib_state), p(o), p(lib_state), None, T, B, H, Hk, K, V,
                         K ** -0.5, 0, p(ws), n, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert rc == 0 and torch.equal(lib_state, want["state"]) and torch.equal(o, want["o"])


def test_empty():
    t = make(3, 2, 2, 1, 8, 8, seed=15)
    e = {k: (v[:0] if k not in ("state0", "grad_state") and v is not None else v) for k, v in t.items()}
    got = run(e)
    assert got["o"].shape == (0, 2, 2, 8) and torch.equal(got["state"], t["state0"])
    assert torch.equal(got["grad_state0"], t["grad_state"])
    e = {k: None if v is None else (v[:, :0] if k not in ("state0", "grad_state") else v[:0]) for k, v in t.items()}
    got = run({k: None if v is None else v.contiguous() for k, v in e.items()})
    assert got["o"].shape == (3, 0, 2, 8) and got["state"].shape == (0, 2, 8, 8)


def test_pieces():
    """A sequence in two calls, the state handed on at a border of chunks: the bits of one call."""
    t = make(192, 2, 2, 2, 64, 64, dtype=torch.bfloat16, seed=16)
    inputs = [t[n] for n in ("q", "k", "v", "log_decay", "beta")]
    o, state = lrs.gdr_fwd(*inputs, state0=t["state0"], want_state=True)
    o1, s1 = lrs.gdr_fwd(*[x[:128] for x in inputs], state0=t["state0"], want_state=True)
    o2, s2 = lrs.gdr_fwd(*[x[128:] for x in inputs], state0=s1, want_state=True)
    assert torch.equal(torch.cat([o1, o2]), o) and torch.equal(s2, state)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 1), (5, 3, 3, 20, 33), (7, 4, 2, 64, 64), (4, 2, 1, 128, 128),
                                   (3, 2, 2, 128, 300), (2, 6, 2, 100, 256)])
def test_step(shape, dtype):
    """Single tokens against one step of the plain form; fp32 sums of at most 128 terms."""
    B, H, Hk, K, V = shape
    t = make(1, B, H, Hk, K, V, dtype=dtype, seed=sum(shape))
    ref = reference({**t, "grad_o": None})
    pool = torch.randn(B + 3, H, K, V, device=DEV)
    slots = torch.randperm(B + 3, device=DEV)[:B].int()
    pool[slots.long()] = t["state0"]
    before = pool.clone()
    o = lrs.gdr_step(t["q"][0], t["k"][0], t["v"][0], t["log_decay"][0], t["beta"][0], pool, slots=slots)
    close({"o": o[None], "state": pool[slots.long()]}, ref)
    others = [i for i in range(B + 3) if i not in slots.tolist()]
    assert torch.equal(pool[others], before[others])


def test_step_idle_and_without_slots():
    B, H, K, V = 4, 2, 16, 24
    t = make(1, B, H, H, K, V, seed=3)
    args = [t[n][0] for n in ("q", "k", "v", "log_decay", "beta")]
    pool = torch.randn(5, H, K, V, device=DEV)
    one, two = pool.clone(), pool.clone()
    a = lrs.gdr_step(*args, one)
    b = lrs.gdr_step(*args, two, slots=torch.tensor([0, -1, 2, 5], dtype=torch.int32, device=DEV))
    assert torch.equal(a[[0, 2]], b[[0, 2]]) and (b[[1, 3]] == 0).all()
    assert torch.equal(one[[0, 2]], two[[0, 2]]) and torch.equal(two[[1, 3, 4]], pool[[1, 3, 4]])
    assert torch.equal(one[4], pool[4])


def test_step_continues_a_prompt():
    """A prompt, then single tokens: what the forward gives for the whole sequence."""
    T, B, H, Hk, K, V = 80, 3, 4, 2, 64, 64
    t = make(T, B, H, Hk, K, V, seed=4)
    inputs = [t[n] for n in ("q", "k", "v", "log_decay", "beta")]
    ref = reference({**t, "grad_o": None})
    _, pool = lrs.gdr_fwd(*[x[:70] for x in inputs], state0=t["state0"], want_state=True)
    steps = [lrs.gdr_step(*[x[i] for x in inputs], pool) for i in range(70, T)]
    o = f64(torch.stack(steps))
    assert ((o - ref["o"][70:]).abs() <= FWD * (usual("o", ref["o"]) + ref["o"][70:].abs())).all()
    close({"state": pool}, ref)


def test_repeatable():
    t = make(400, 2, 4, 2, 64, 64, dtype=torch.bfloat16, seed=17, resets=0.01)
    runs = [run(t) for _ in range(3)]
    for r in runs[1:]:
        for name in r:
            assert torch.equal(r[name], runs[0][name]), name


def test_refusals():
    t = make(4, 2, 4, 2, 16, 16)
    q, k, v, g, b = (t[n] for n in ("q", "k", "v", "log_decay", "beta"))
    with pytest.raises(TypeError):
        lrs.gdr_fwd(q.half(), k.half(), v.half(), g, b)
    with pytest.raises(TypeError):
        lrs.gdr_fwd(q, k.bfloat16(), v, g, b)
    with pytest.raises(TypeError):
        lrs.gdr_fwd(q, k, v, g.bfloat16(), b)
    with pytest.raises(TypeError):
        lrs.gdr_fwd(q, k, v, None, b)
    with pytest.raises(ValueError):
        lrs.gdr_fwd(q, k, v[:, :, :3].contiguous(), g[:, :, :3].contiguous(), b[:, :, :3].contiguous())
    with pytest.raises(ValueError):
        lrs.gdr_fwd(q[..., :8], k, v, g, b)
    with pytest.raises(ValueError):
        lrs.gdr_fwd(q.transpose(0, 1), k.transpose(0, 1), v.transpose(0, 1), g, b)
    with pytest.raises(ValueError):
        lrs.gdr_fwd(q.transpose(2, 3), k, v, g, b)
    with pytest.raises(ValueError):
        lrs.gdr_fwd(q, k, v, g, b, state0=t["state0"][:1])
    with pytest.raises(lrs.LrsError):
        lrs.gdr_fwd(q, k, v, g, b, scale=math.nan)
    with pytest.raises(lrs.LrsError):
        lrs.gdr_fwd(q, k, v, g, b, out=v)
    with pytest.raises(TypeError):
        lrs.gdr_bwd(q, k, v, g, b, None, t["grad_o"])
    big = make(2, 1, 1, 1, 129, 8)
    with pytest.raises(lrs.LrsError):
        lrs.gdr_fwd(*[big[n] for n in ("q", "k", "v", "log_decay", "beta")])
    with pytest.raises(ValueError):
        lrs.gdr_step(q[0], k[0], v[0], g[0], b[0], t["state0"][:1])
    ck = lrs.gdr_checkpoints(k, v)
    with pytest.raises(ValueError):
        lrs.gdr_bwd(q, k, v, g, b, ck, t["grad_o"], grad_qkv=(torch.empty_like(v), k, v))
    with pytest.raises(lrs.LrsError):  # a gradient over an input
        lrs.gdr_bwd(q, k, v, g, b, ck, t["grad_o"], grad_qkv=(q, torch.empty_like(k), torch.empty_like(v)))
