"""The delta rule's chains with one, two and four blocks of 16 columns a workgroup, which the
number of heads decides (256 compute units); blocks that are partly or wholly past V, both
widths of K, restarts inside chunks.  Bounds: those of test_gpu_gdr."""
import pytest
import torch

import test_gpu_gdr as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,H,Hk,K,V", [(2, 3, 3, 40, 33), (2, 4, 2, 100, 65),   # one
                                        (6, 10, 5, 40, 72), (4, 16, 16, 128, 128), (1, 200, 100, 66, 17),  # two
                                        (13, 10, 5, 40, 72), (10, 13, 13, 72, 66), (4, 66, 6, 128, 20)])  # four
@pytest.mark.parametrize("resets", [0.0, 0.03])
def test_blocks(B, H, Hk, K, V, resets, dtype):
    t = G.make(130, B, H, Hk, K, V, dtype, seed=B + V, resets=resets)
    G.close(G.run(t), G.reference(t))


@pytest.mark.parametrize("T", [1, 63, 64, 65, 128, 129, 192])
@pytest.mark.parametrize("K", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_few_chunks(T, K, dtype):
    """Operands are brought in one and two chunks ahead: sequences shorter than that."""
    t = G.make(T, 2, 2, 1, K, 40, dtype, seed=T)
    G.close(G.run(t), G.reference(t))
    G.close(G.run(t, train=False), G.reference(t))
