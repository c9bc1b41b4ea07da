"""CPU: the interface to the recurrence's waits."""
import ctypes

import pytest
import torch

import stacked_lstm_forward_amd as sl
from stacked_lstm_forward_amd import block

from .test_block import FAKE, glr_desc


def test_last_error_refuses():
    d = glr_desc()
    for train in (False, True):
        assert block.lstm_glr_last_error(None, train, FAKE, 0) == sl.LSTM_ERR_INVALID_ARG
        assert block.lstm_glr_last_error(glr_desc(T=0), train, FAKE, 0) == sl.LSTM_ERR_INVALID_ARG
        for ws in (None, FAKE + 64):
            assert block.lstm_glr_last_error(d, train, ws, 0) == sl.LSTM_ERR_WORKSPACE
    with pytest.raises(ValueError):
        x = torch.zeros(2, 3, 8)
        block.prepare_glr(x, x).last_error()


@pytest.mark.parametrize("us", [0, 1, -1, 1 << 40, (1 << 63) - 1, -(1 << 63)])
def test_any_limit_is_a_description(us):
    d = glr_desc(T=100000, wait_timeout_us=us)
    assert block.lstm_glr_validate(d) == block.lstm_glr_validate(d, True) == sl.LSTM_OK
    assert block.lstm_glr_workspace_size(d) == block.lstm_glr_workspace_size(glr_desc(T=100000))


def test_the_limit_is_the_descriptions_last_field():
    assert block.GlrDesc.wait_timeout_us.offset == ctypes.sizeof(block.GlrDesc) - 8 == 24 + 8 * 16
