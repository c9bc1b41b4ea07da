"""GPU: a clipping problem whose tensors change at their address leaves the memory behind them alone."""
import pytest
import torch

from stacked_lstm_forward_amd import block

from .test_gpu_block import DEV

pytestmark = pytest.mark.gpu


def test_clip_of_a_tensor_that_shrank_at_its_address():
    flat = torch.full((10000,), 3.0, device=DEV)
    t = flat[:6000]
    p = block.prepare_clip([t], 1.0)
    first = t.data
    t.data = flat[:5000]
    with pytest.raises(ValueError):
        p.run()
    torch.cuda.synchronize()
    assert bool((flat == 3.0).all())
    t.data = first
    p.run()
    assert abs(float(p.norm) / (3 * 6000 ** 0.5) - 1) < 1e-6
    assert bool((flat[6000:] == 3.0).all()) and bool((flat[:6000] < 0.1).all())


def test_clip_follows_many_tensors_to_other_memory():
    t = [torch.full((i % 7 + 1,), 1.0, device=DEV) for i in range(300)]
    p = block.prepare_clip(t, float("inf"))
    n = sum(x.numel() for x in t)
    for value in (1.0, 2.0, 5.0):
        for x in t[::3]:
            x.data = torch.full_like(x, value)
        p.run()
        want = sum(x.numel() * (value ** 2 if i % 3 == 0 else 1.0) for i, x in enumerate(t)) ** 0.5
        assert abs(float(p.norm) / want - 1) < 1e-6
    assert n == sum(x.numel() for x in t)
