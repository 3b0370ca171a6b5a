"""The gradient of the delta rule's log decay where it is small beside what it is taken from:
heads that decay strongly, and single strong steps among weak ones.

Bounds: those of test_gpu_gdr, 1.2e-4 of the usual size.  At step t the gradient is a sum of
products that all pass through step t, each with its decay as a factor; pairs of steps on the
same side of t have no part in it, however large they are.  So the bound holds beside the root
mean square of the head's own gradients, and, for the strong steps of a head, beside that of
the gradients at those steps alone."""
import pytest
import torch

import test_gpu_gdr as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,resets,state", [(64, 0.0, False), (64, 0.0, True), (130, 0.0, True), (200, 0.05, True)])
@pytest.mark.parametrize("K,V", [(64, 64), (100, 40)])
def test_heads_that_decay_strongly(T, resets, state, K, V, dtype):
    decays = torch.tensor([-1.0, -4.0, -8.0, -12.0, -16.0, -20.0], device=G.DEV)
    t = G.make(T, 2, 6, 2, K, V, dtype, seed=T + K, resets=resets, state=state)
    t["log_decay"] = decays.expand(T, 2, 6).contiguous()
    G.close(G.run(t), G.reference(t))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("strong", [-8.0, -16.0])
@pytest.mark.parametrize("at", [[30], [0, 64], [63, 127], [5, 21, 40, 77, 100, 128]])
def test_strong_steps_among_weak_ones(at, strong, dtype):
    t = G.make(130, 2, 4, 2, 64, 48, dtype, seed=len(at))
    t["log_decay"] *= 0.1
    t["log_decay"][at] = strong
    got, ref = G.run(t), G.reference(t)
    G.close(got, ref)
    x, y = G.f64(got["grad_log_decay"])[at], ref["grad_log_decay"][at]
    size = y.square().mean(0, keepdim=True).sqrt()
    assert ((x - y).abs() <= G.BWD * (size + y.abs())).all(), float(((x - y).abs() / (size + y.abs())).max())
