"""The layer norm's gradients of gamma and beta over very many rows.

Bound: 1e-5 of the sum of the absolute terms.  A workgroup adds at most 256 rows in
fp32 before fp64 takes over: 256 * 2^-25 = 8e-6 at the very worst."""
import pytest
import torch

import linear_recurrence_scan_diagonal_amd as lrs

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("R,D,dtype", [(16_000_000, 64, torch.bfloat16), (3_000_000, 1200, torch.bfloat16),
                                       (2_000_000, 1028, torch.float32), (1_500_000, 4100, torch.float32)])
def test_sums_over_millions_of_equal_rows(R, D, dtype):
    """Equal terms of one sign are rounded the same way at every step: a running fp32
    sum of 4000 of them would be off by up to 6e-5."""
    g = torch.Generator().manual_seed(D)
    row = torch.randn(D, generator=g).to(dtype).to(DEV)
    grad = (torch.rand(D, generator=g) + 0.5).to(dtype).to(DEV)
    gamma = torch.ones(D, device=DEV)
    x = row.expand(R, D).contiguous()
    gy = grad.expand(R, D).contiguous()
    mean, rstd = (v.expand(R).contiguous() for v in lrs.layernorm_fwd(row[None], gamma, save=True)[2:])
    _, gg, gb = lrs.layernorm_bwd(x, gamma, mean, rstd, gy)
    # the terms as fp32 has them; their own rounding is not what this is about
    xh = (row.float() - mean[0]) * rstd[0]
    for got, term in ((gg, grad.double() * xh.double()), (gb, grad.double())):
        off = ((got.double() - R * term).abs() / (R * term.abs())).max()
        assert off <= 1e-5, off
