"""GPU: a wait of the recurrence that passes its limit is reported, and the kernel exits normally."""
import pytest
import torch

import stacked_lstm_forward_amd as sl
from stacked_lstm_forward_amd import block

from .test_gpu_block_limits import bits, glr_problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forced_wait_timeout(dtype):
    """A negative limit fails every wait that is not satisfied at its first look; the next call is clean and right."""
    p, up, names = glr_problem(4, 16384, 256, dtype=dtype)  # 32 and more chunks, the groups' states after one another
    p.forward()
    assert p.last_error() == sl.LSTM_OK
    p.backward(*up)
    assert p.last_error(train=True) == sl.LSTM_OK
    want = [bits(getattr(p, n)).clone() for n in names]
    p.desc.wait_timeout_us = -1
    p.forward()
    assert p.last_error() == sl.LSTM_ERR_BARRIER_TIMEOUT
    assert bool(p.y.isnan().any())
    p.desc.wait_timeout_us = 0
    p.forward()
    assert p.last_error() == sl.LSTM_OK
    p.desc.wait_timeout_us = -1
    p.backward(*up)
    assert p.last_error(train=True) == sl.LSTM_ERR_BARRIER_TIMEOUT
    assert bool(p.df.isnan().any())
    p.desc.wait_timeout_us = 10000000
    p.backward(*up)
    assert p.last_error(train=True) == sl.LSTM_OK
    for n, w in zip(names, want):
        assert torch.equal(bits(getattr(p, n)), w), n


@pytest.mark.parametrize("T", [1, 40, 500])
def test_calls_without_waits_report_none(T):
    """Whatever the workspace holds: a sentence of one chunk has no error word."""
    p, up, _ = glr_problem(2, T, 64, dtype="bf16")
    p.desc.wait_timeout_us = -1
    p.ws.fill_(255)
    p.forward()
    waits = block.lstm_glr_workspace_size(p.desc) > 256
    if not waits:
        assert p.last_error() == sl.LSTM_OK
        p.ws.fill_(255)
        p.backward(*up)
        assert p.last_error(train=True) == sl.LSTM_OK
    assert waits == (T == 500)
