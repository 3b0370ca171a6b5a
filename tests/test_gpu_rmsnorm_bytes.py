"""The 8-bit output of the RMS norm at the borders between two bytes: exactly the quotient
y / scale in fp32, rounded to nearest, ties to even, with y the fp32 output of rmsnorm_fwd for
the same rows.  No tolerance: a quotient of two fp32 numbers in fp64, rounded to fp32, is the
fp32 quotient (53 bits are more than twice 24 and two)."""
import pytest
import torch

import linear_recurrence_scan_diagonal_amd as lrs
import block_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def exact(x, gamma, group):
    q, scales, _ = lrs.rmsnorm_fwd_fp8(x, gamma, group=group)
    y = lrs.rmsnorm_fwd(x, gamma)[0]
    rows, D = x.shape
    step = group or D
    for i in range(scales.shape[1]):
        part = y[:, i * step:(i + 1) * step]
        top = part.abs().amax(1).double()
        scale = torch.where(top == 0, 1.0, (top / 448).float().clamp(min=2.0 ** -120).double()).float()
        assert torch.equal(scales[:, i], scale)
        want = (part.double() / scale[:, None].double()).float().to(torch.float8_e4m3fn)
        have = q[:, i * step:(i + 1) * step]
        off = want.view(torch.uint8) != have.contiguous().view(torch.uint8)
        assert not off.any(), (int(off.sum()), part[off][:4].tolist(), scale[off.any(1)][:4].tolist())


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("D", [128, 100, 300, 2048, 5000, 20000])
@pytest.mark.parametrize("size", [1.0, 1e30, 1e-30, 2.0 ** -112])
def test_at_the_borders(D, size, group):
    """Rows whose quotients lie within three steps of fp32 from a border."""
    grid = R.e4m3_grid()
    borders = (grid[1:] + grid[:-1]) / 2
    g = torch.Generator().manual_seed(D)
    rows = 400
    b = borders[torch.randint(0, len(borders), (rows, D), generator=g)]
    x = b * (1 + torch.randint(-3, 4, (rows, D), generator=g) * 2.0 ** -24) * torch.where(torch.rand(rows, D, generator=g) < 0.5, -1, 1)
    x[:, ::128 if group else D] = 448.0
    x *= 1 + torch.rand(rows, 1, generator=g)
    exact(x.float().to(DEV), torch.full((D,), size, device=DEV), group)


@pytest.mark.parametrize("group", [0, 128])
def test_many_values(group):
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(1 << 14, 1024, generator=g, device=DEV)
    exact(x, 1 + 0.2 * torch.randn(1024, generator=g, device=DEV), group)
