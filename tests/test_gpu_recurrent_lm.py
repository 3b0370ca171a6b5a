"""The example model end to end: its gradients against a plain form in 64 bits, a
few training steps, and decoding against the forward over the whole sequence."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "recurrent_lm", os.path.join(ROOT, "examples", "recurrent_lm.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def plain_loss(params, tokens, targets, reset, blocks):
    """The model's loss from its formulas, in the parameters' type."""
    def norm(s, gamma, beta):
        mean = s.mean(-1, keepdim=True)
        var = ((s - mean) ** 2).mean(-1, keepdim=True)
        return (s - mean) / torch.sqrt(var + 1e-5) * gamma + beta
    w = params["embedding"]
    stream = w[tokens]
    for i in range(blocks):
        p = {k.split(".")[2]: v for k, v in params.items() if k.startswith(f"blocks.{i}.")}
        zr, zi, x = (norm(stream, p["gamma"], p["beta"]) @ p["project"].t()).chunk(3, dim=-1)
        la = -8.0 * torch.nn.functional.softplus(p["decay"]) * torch.sigmoid(zr + p["bias_r"])
        a, m = torch.exp(la), torch.sqrt(-torch.expm1(2 * la))
        start = reset[..., None]
        a, m = torch.where(start, 0.0, a), torch.where(start, 1.0, m)
        u = m * torch.sigmoid(zi + p["bias_i"]) * x
        h, rows = torch.zeros_like(u[0]), []
        for t in range(u.shape[0]):
            h = a[t] * h + u[t]
            rows.append(h)
        stream = stream + torch.stack(rows) @ p["back"].t()
    logits = (norm(stream, params["gamma"], params["beta"]) @ w.t()).flatten(0, 1)
    keep = targets.flatten() >= 0
    lse = torch.logsumexp(logits[keep], -1)
    return (lse - logits[keep, targets.flatten()[keep]]).mean()


def test_gradients(example):
    """fp32 model, all parameters.  The operators are good to about 1e-6 of the
    largest value each; the model chains some twenty of them and torch's fp32
    products, so 1e-4 of a gradient's largest value leaves a wide margin, while a
    missing term (a residual's gradient, a restart) shows at 1e-2 or more."""
    torch.manual_seed(3)
    gen = torch.Generator().manual_seed(4)
    tokens, targets, reset = example.documents(37, 5, 19, 3, 14, gen)
    model = example.RecurrentLM(19, 24, 2, torch.float32)
    loss = model.loss(tokens.cuda(), targets.cuda(), reset.cuda())
    (3.0 * loss).backward()
    params = {k: v.detach().double().cpu().requires_grad_() for k, v in model.named_parameters()}
    ref = plain_loss(params, tokens, targets, reset, 2)
    (3.0 * ref).backward()
    loss, ref = float(loss.detach()), float(ref.detach())
    assert abs(loss - ref) < 1e-5 * abs(ref)
    for k, v in model.named_parameters():
        want = params[k].grad
        top = float(want.abs().max())
        assert top > 0, k
        assert float((v.grad.double().cpu() - want).abs().max()) < 1e-4 * top, k


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_trains(example, dtype):
    """Loss falls well below that of a uniform guess, log 32 = 3.47."""
    torch.manual_seed(5)
    gen = torch.Generator().manual_seed(6)
    model = example.RecurrentLM(32, 64, 2, dtype)
    losses = example.train(
        model, 120, lambda: [t.cuda() for t in example.documents(64, 32, 32, 3, 32, gen)], lr=5e-3)
    assert 3.0 < losses[0] < 8.0
    assert losses[-1] < 1.0


@pytest.mark.parametrize("dtype, tol", [(torch.float32, 1e-4), (torch.bfloat16, 0.1)])
def test_decoding_is_the_forward(example, dtype, tol):
    """A prompt and single steps give the logits of one prompt over all tokens, also
    with an idle sequence in the batch and rows of the pool out of order.  The
    logits are about 1 in size; bf16 rounds each of some ten values on the way to
    2^-9 of itself."""
    torch.manual_seed(7)
    model = example.RecurrentLM(50, 40, 3, dtype)
    tokens = torch.randint(0, 50, (21, 4), device="cuda")
    slots = torch.tensor([6, 0, 3, 1], dtype=torch.int32, device="cuda")
    decoder, whole = example.Decoder(model, 7), example.Decoder(model, 7)
    decoder.prompt(tokens[:9], slots)
    busy = torch.tensor([6, 0, -1, 1], dtype=torch.int32, device="cuda")
    for t in range(9, 21):
        got = decoder.step(tokens[t], busy)
        want = whole.prompt(tokens[:t + 1], slots)
        for b in (0, 1, 3):
            assert float((got[b].float() - want[b].float()).abs().max()) < tol, (t, b)
    for i in range(3):
        for b in (0, 1, 3):
            row = int(slots[b])
            assert float((decoder.pool[i][row] - whole.pool[i][row]).abs().max()) < tol, (i, b)
        # the idle sequence's state is the prompt's
        first = example.Decoder(model, 7)
        first.prompt(tokens[:9], slots)
        assert torch.equal(decoder.pool[i][3], first.pool[i][3])
