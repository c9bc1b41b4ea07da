"""Layer norm on the GPU: the mean of rows that are large against their spread."""
import math

import pytest
import torch

from stacked_lstm_forward_amd import block

from .block_reference import W
from .test_gpu_block import DEV, DT, Make

pytestmark = pytest.mark.gpu

WIDTHS = [1, 5, 20, 33, 100, 300, 500, 777, 1000, 1025, 2000, 3001, 4500, 9001, 16383]  # one lane to sixteen waves


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", WIDTHS)
def test_norm_of_rows_of_one_value(N, dtype):
    """Whatever the value: its mean is itself, nothing is left to be normalised, and rstd is 1 / sqrt(eps)."""
    g = torch.Generator().manual_seed(N)
    v = (torch.rand(1, 99, 1, generator=g) * 9e4 + 1e4) * torch.where(torch.rand(1, 99, 1, generator=g) < 0.5, -1.0, 1.0)
    v = torch.cat((v, torch.full((1, 1, 1), 12345.678)), 1).to(DT[dtype])
    x = v.expand(1, 100, N).contiguous().to(DEV)
    w, b = (torch.randn(N, generator=g).to(DT[dtype]).to(DEV) for _ in range(2))
    for eps in (1e-5, 1e-12):
        p = block.prepare_norm(x, w, b, train=True, eps=eps)
        p.forward()
        assert torch.equal(p.mean.cpu(), v[..., 0].float())
        assert torch.equal(p.y, b.expand(1, 100, N))
        want = 1 / math.sqrt(float(torch.tensor(eps)))
        assert float((p.rstd - want).abs().max()) <= 4 * W * want
        p.backward(torch.ones_like(x, dtype=torch.float32))
        assert not p.dw.any() and bool(torch.isfinite(p.dx).all())


@pytest.mark.parametrize("N", WIDTHS[4:])
@pytest.mark.parametrize("mean,spread", [(3e4, 1.0), (-1e3, 1e-2), (7.0, 1e-5)])
def test_norm_of_rows_far_from_zero(mean, spread, N):
    m = Make(2, 50, "bth", N)
    x = m.seq(N, "f32", spread, mean)
    p = block.prepare_norm(x, train=True, eps=1e-12)
    p.forward()
    s = x.cpu().double()
    mu = s.mean(-1, keepdim=True)
    d = s - mu
    # the sum of the distances to a first mean corrects it (80 roundings of their magnitude, which is the spread and
    # what that mean is off by: no more than 80 W of the values); then the waves' means and the row's are rounded once
    far = d.abs().mean(-1, keepdim=True)
    off = 2 * W * mu.abs() + 80 * W * (far + 80 * W * mu.abs())
    assert bool(((p.mean.cpu().double()[..., None] - mu).abs() <= off).all())
    var = d.square().mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(var + 1e-12)
    rel = 0.5 * (2 * far * off + off ** 2) / (var + 1e-12) + 90 * W
    assert bool(((p.rstd.cpu().double()[..., None] - rstd).abs() <= rel * rstd).all())
    assert bool(((p.y.cpu().double() - d * rstd).abs() <= (off + d.abs() * (rel + 4 * W)) * rstd * (1 + rel)).all())


@pytest.mark.parametrize("N", [100, 1000, 3001])
def test_norm_of_rows_that_are_not_finite(N):
    """An infinity or a NaN stays in its row; the mean says which."""
    x = torch.randn(1, 4, N, generator=torch.Generator().manual_seed(1))
    for t, bad in enumerate((math.inf, -math.inf, math.nan)):
        x[0, t, N // 2] = bad
    p = block.prepare_norm(x.to(DEV), train=True)
    p.forward()
    assert p.mean[0, :2].tolist() == [math.inf, -math.inf] and bool(p.mean[0, 2].isnan())
    assert bool(p.y[0, :3].isnan().all()) and bool(p.y[0, 3].isfinite().all())
