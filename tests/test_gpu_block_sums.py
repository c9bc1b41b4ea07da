"""GPU: the weight gradients' sums over many rows are taken in parts, not one row after the other."""
import pytest
import torch

from stacked_lstm_forward_amd import block

from .block_reference import W
from .test_gpu_block import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [16, 200, 512, 1500, 5000])
def test_norm_weight_gradients_of_many_rows(N):
    """A group of lanes adds at most rows / 256 rows one after the other where a row takes a workgroup, fewer where it
    takes less; then 6 steps of groups and waves, and the workgroups' sums in parts of 3 and 8 and over 32 lanes."""
    B, T = 8, 2000000 // N
    rows = B * T
    x = torch.randn(B, T, N, generator=torch.Generator().manual_seed(N)).to(DEV)
    dy = torch.full_like(x, 0.1)
    p = block.prepare_norm(x, torch.ones(N, device=DEV), torch.zeros(N, device=DEV), train=True)
    p.forward()
    p.backward(dy)
    want = rows * float(dy[0, 0, 0])
    roundings = rows / 256 + 30
    assert float((p.db.double() - want).abs().max()) <= roundings * W * want
    n = (x.double() - p.mean.double()[..., None]) * p.rstd.double()[..., None]
    terms = n * float(dy[0, 0, 0])
    off = (p.dw.double() - terms.sum((0, 1))).abs()
    assert bool((off <= (roundings + 3) * W * terms.abs().sum((0, 1))).all())  # (a term: 3 roundings)
