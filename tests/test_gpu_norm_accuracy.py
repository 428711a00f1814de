"""Layer norm where its statistics have no roundings to hide behind: sums that fp32 holds exactly."""
import pytest
import torch

import block_ref as R
import convolution_nhwc_implicit_amd as nn

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("d", [2, 16, 131, 512, 1001, 4096, 8190, 16384])
def test_small_deviations_around_a_large_mean(d, residual):
    """Deviations of 2^-4 around 64, as many up as down and none at an odd one: every partial sum is a multiple of 2^-4 up
    to 64 d, 24 bits at most, so mean, deviations and the sum of their squares are exact. What is left is a quotient, the
    root, its inverse, two products and a sum: 8 roundings of 2^-24. Mean squares less the squared mean would be off by some
    steps of 4096 in fp32, 2^-12, of a variance of 2^-8."""
    g = torch.Generator().manual_seed(d)
    sign = torch.cat([torch.ones(d // 2), -torch.ones(d // 2), torch.zeros(d % 2)])
    sign = torch.stack([sign[torch.randperm(d, generator=g)] for _ in range(4)])
    x = 64.0 + sign * 2.0 ** -4
    w, b = 1.0 + 0.25 * torch.rand(d, generator=g), torch.rand(d, generator=g)
    res = torch.randint(-20, 20, x.shape, generator=g) * 2.0 ** -4 if residual else None
    y = nn.layer_norm((x - res if residual else x).to(DEV), w.to(DEV), b.to(DEV), eps=0.0, residual=res.to(DEV) if residual else None)
    if residual:
        y, total = y
        assert torch.equal(total.cpu(), x)
    s, wd, bd = sign.double(), w.double(), b.double()
    xh = s * (d / (d - d % 2)) ** 0.5
    assert bool(((y.double().cpu() - (xh * wd + bd)).abs() <= 8 * R.U * (wd + bd) * 1.01).all())
    dy = torch.randn(4, d, generator=g)
    k = nn.layer_norm_grad(dy.to(DEV), x.to(DEV), w.to(DEV), b.to(DEV), eps=0.0)
    gw = dy.double() * wd
    rstd = 16 * (d / (d - d % 2)) ** 0.5
    want = rstd * (gw - gw.mean(1, keepdim=True) - xh * (gw * xh).mean(1, keepdim=True))
    # two sums over the row
    tol = 2 * R.ADDS * R.U * rstd * (gw.abs() + gw.abs().mean(1, keepdim=True) + xh.abs() * (gw * xh).abs().mean(1, keepdim=True))
    assert bool(((k["dx"].double().cpu() - want).abs() <= tol).all())
    # four terms each, of 8 roundings
    for got, terms in ((k["dw"], dy.double() * xh), (k["db"], dy.double())):
        assert bool(((got.double().cpu() - terms.sum(0)).abs() <= 12 * R.U * terms.abs().sum(0)).all())
