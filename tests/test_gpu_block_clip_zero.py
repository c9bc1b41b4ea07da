"""GPU: gradients that are all 0 stay 0, whatever the limit."""
import pytest
import torch

from stacked_lstm_forward_amd import block

from .test_gpu_block import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit", [0.0, 1.0, float("inf")])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("sizes", [[5000, 3], [0]], ids=str)
def test_clip_of_nothing(sizes, eps, limit):
    t = [torch.zeros(n, device=DEV) for n in sizes]
    out = [torch.full_like(x, float("nan")) for x in t]
    p = block.prepare_clip(t, limit, out=out, eps=eps)
    p.run()
    assert float(p.norm) == 0 and float(p.coef) == (0.0 if limit == 0 and eps > 0 else 1.0)
    assert not any(bool(x.any()) for x in out)


def test_clip_to_nothing():
    t = torch.tensor([3.0, -4.0], device=DEV)
    p = block.prepare_clip([t], 0.0, eps=0.0)
    p.run()
    assert float(p.norm) == 5 and float(p.coef) == 0 and not t.any()
