"""CPU tests of the decoder operators' limits and refusals (host checks; nothing is launched)."""
import pytest

import stacked_lstm_forward_amd as sl
from stacked_lstm_forward_amd import decoder

from .test_decoder import FAKE, desc

MOST = (1 << 31) - 4096  # rows of all heads, keys of all sentences: the kernels' 32-bit counters step past them


@pytest.mark.parametrize("change", [dict(B=1, S=1), dict(B=1, Tq=1), dict(B=2, S=2), dict(B=2, Tq=2)], ids=str)
def test_lengths_leave_room_for_the_kernels_counters(change):
    axis = "S" if "S" in change else "Tq"

    def at(n):
        return desc(**{**dict(B=1, Tq=1, S=1, Hq=1, Hkv=1, D=8), **change, axis: n})

    n = MOST // change["B"]
    assert decoder.lstm_attn_validate(at(n)) == sl.LSTM_OK
    assert decoder.lstm_attn_workspace_size(at(n)) > 0
    for more in (n + 1, (1 << 31) // change["B"] - 200, (1 << 31) // change["B"] - 1):
        d = at(more)
        for train in (False, True):
            assert decoder.lstm_attn_validate(d, train) == sl.LSTM_ERR_UNSUPPORTED
        assert decoder.lstm_attn_workspace_size(d) == 0 and decoder.lstm_attn_bwd_workspace_size(d) == 0
        assert decoder.lstm_attn_fwd(d, *[FAKE] * 3, None, None, *[FAKE] * 3, stream=0) == sl.LSTM_ERR_UNSUPPORTED


def test_the_longest_key_axis_is_split():
    # two sums of D = 8 and two statistics a part and row: more than the least workspace
    d = desc(B=1, Tq=1, S=MOST, Hq=1, Hkv=1, D=8)
    assert decoder.lstm_attn_workspace_size(d) > 200 * (8 + 2) * 4


def test_gradients_count_their_workgroups():
    d = desc(B=1 << 30, Tq=1, S=1, Hq=1, Hkv=1, D=8)  # a tile of rows and one of keys for each sentence: 2^31
    assert decoder.lstm_attn_validate(d) == sl.LSTM_OK
    assert decoder.lstm_attn_validate(d, train=True) == sl.LSTM_ERR_UNSUPPORTED
    assert decoder.lstm_attn_bwd_workspace_size(d) == 0
    d = desc(B=(1 << 30) - 2048, Tq=1, S=1, Hq=1, Hkv=1, D=8)
    assert decoder.lstm_attn_validate(d, train=True) == sl.LSTM_OK
