"""CPU tests of the decoder operators' limits and refusals (host checks; nothing is launched)."""
import pytest
import torch

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


# ---- problems ------------------------------------------------------------------


def attn_problem(train=True):
    q, k = torch.zeros(2, 3, 4, 64), torch.zeros(2, 5, 2, 64)
    return decoder.prepare_attn(q, k, k.clone(), kv_len=torch.zeros(2, dtype=torch.int32), train=train)


def beam_problem():
    return decoder.prepare_beam(torch.zeros(2, 4, 50), torch.zeros(2, 4), torch.zeros(2, 4, dtype=torch.uint8),
                                torch.zeros(2, 4, dtype=torch.int32), eos=2,
                                states=(torch.zeros(1, 8, 8), torch.zeros(1, 8, 8)))


def test_problems_in_host_memory_do_not_run():
    p, s = attn_problem(), beam_problem()
    for stream in (None, 0):
        with pytest.raises(ValueError):
            p.forward(stream=stream)
        with pytest.raises(ValueError):
            p.backward(torch.zeros(2, 3, 4, 64), stream=stream)
        with pytest.raises(ValueError):
            s.step(stream=stream)


@pytest.mark.parametrize("name,value,error", [
    ("q", torch.zeros(2, 3, 4, 32), ValueError), ("k", torch.zeros(2, 4, 2, 64), ValueError),
    ("v", torch.zeros(2, 5, 2, 64, dtype=torch.bfloat16), TypeError),
    ("v", torch.zeros(2, 5, 2, 65)[..., 1:], ValueError), ("o", torch.zeros(2, 3, 4, 64, device="meta"), ValueError),
    ("dk", torch.zeros(2, 5, 64, 2).transpose(2, 3), ValueError), ("kv_len", torch.zeros(1, dtype=torch.int32), ValueError),
    ("kv_len", torch.zeros(2, dtype=torch.int64), TypeError), ("kv_len", torch.zeros(4, dtype=torch.int32)[::2], ValueError),
    ("key_mask", torch.zeros(2, 4, dtype=torch.bool), ValueError), ("key_mask", torch.zeros(2, 5), TypeError),
    ("lse", torch.zeros(2, 4, 2), ValueError), ("ws", torch.zeros(8, dtype=torch.uint8), ValueError),
    ("bws", torch.zeros(1 << 12, dtype=torch.uint8)[1:], ValueError),
])
def test_what_replaces_a_tensor_of_an_attention_problem_is_checked(name, value, error):
    p = attn_problem()
    before = getattr(p, name)
    with pytest.raises(error):
        setattr(p, name, value)
    assert getattr(p, name) is before


def test_tensors_of_an_attention_problem_may_be_replaced():
    p = attn_problem()
    q = torch.zeros(3, 2, 4, 64).transpose(0, 1)  # another layout: its strides are the description's
    p.q = q
    assert p.q is q and (p.desc.q.b, p.desc.q.t, p.desc.q.h) == q.stride()[:3]
    p.kv_len, p.lse = None, None
    p.kv_len, p.lse = torch.ones(2, dtype=torch.int32), torch.zeros(2, 4, 3)
    p.key_mask = torch.ones(2, 5, dtype=torch.bool)
    assert p.key_mask.dtype == torch.uint8
    p = attn_problem(train=False)
    with pytest.raises(ValueError):
        p.dq = torch.zeros(2, 3, 4, 64)


def test_what_the_rounding_of_o_leaves_has_a_place_of_its_own():
    assert attn_problem().o_rest is None and not attn_problem().desc.o_rest  # fp32
    q, k = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 5, 2, 64, dtype=torch.bfloat16)
    assert decoder.prepare_attn(q, k, k).o_rest is None
    p = decoder.prepare_attn(q, k, k, train=True)
    assert p.o_rest.numel() == p.o.numel() and p.desc.o_rest == p.o_rest.data_ptr()
    p.o_rest = None
    assert not p.desc.o_rest
    for bad, error in ((torch.zeros(2, 3, 4, 32, dtype=torch.bfloat16), ValueError), (torch.zeros(2, 3, 4, 64), TypeError)):
        with pytest.raises(error):
            p.o_rest = bad
    d = desc(o_rest=FAKE + 8)
    assert decoder.lstm_attn_fwd(d, *[FAKE] * 3, None, None, *[FAKE] * 3, stream=0) == sl.LSTM_ERR_UNSUPPORTED
    assert decoder.lstm_attn_bwd(d, *[FAKE] * 3, None, None, *[FAKE] * 7, stream=0) == sl.LSTM_ERR_UNSUPPORTED


@pytest.mark.parametrize("name,value,error", [
    ("logits", torch.zeros(2, 4, 49), ValueError), ("logits", torch.zeros(2, 4, 50, dtype=torch.bfloat16), TypeError),
    ("logits", torch.zeros(2, 50, 4).transpose(1, 2), ValueError), ("scores", torch.zeros(2, 3), ValueError),
    ("scores_out", torch.zeros(2, 4, dtype=torch.float64), TypeError), ("finished", torch.zeros(2, 4), TypeError),
    ("lengths", torch.zeros(4, 2, dtype=torch.int32).t(), ValueError), ("tokens", torch.zeros(2, 4), TypeError),
    ("parents", torch.zeros(1, 4, dtype=torch.int32), ValueError),
    ("states", (torch.zeros(1, 7, 8), torch.zeros(1, 8, 8)), ValueError), ("states", (torch.zeros(1, 8, 8),), ValueError),
    ("states_out", (torch.zeros(1, 8, 8), torch.zeros(1, 8, 8, dtype=torch.bfloat16)), TypeError),
    ("ws", torch.zeros(8, dtype=torch.uint8), ValueError),
])
def test_what_replaces_a_tensor_of_a_beam_problem_is_checked(name, value, error):
    s = beam_problem()
    before = getattr(s, name)
    with pytest.raises(error):
        setattr(s, name, value)
    assert getattr(s, name) is before


def test_tensors_of_a_beam_problem_may_be_replaced():
    s = beam_problem()
    s.logits = torch.zeros(2, 4, 60)[..., 3:53]
    assert s.desc.logits_stride == 60
    s.finished = torch.zeros(2, 4, dtype=torch.bool)
    assert s.finished.dtype == torch.uint8
    s.states, s.states_out = s.states_out, s.states
    before = s.scores, s.states
    s.advance()
    assert s.scores_out is before[0] and s.states_out is before[1]


# ---- alignment -----------------------------------------------------------------


def test_attention_refuses_lengths_and_statistics_that_are_not_aligned():
    d = desc()
    ok = [FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE]
    train = [FAKE, FAKE, FAKE, FAKE, None] + [FAKE] * 7
    for i in (3, 6):  # kv_len, lse
        for by in (1, 2, 3):
            assert decoder.lstm_attn_fwd(d, *[FAKE + by if j == i else x for j, x in enumerate(ok)], stream=0) == \
                sl.LSTM_ERR_INVALID_ARG
            assert decoder.lstm_attn_bwd(d, *[FAKE + by if j == i else x for j, x in enumerate(train)], stream=0) == \
                sl.LSTM_ERR_INVALID_ARG


# ---- scale ---------------------------------------------------------------------


def test_scales_that_fp32_does_not_hold_are_refused():
    # times log2(e) they are infinite, and a score of 0 would be NaN
    for scale in (2.4e38, 3.4e38):
        assert decoder.lstm_attn_validate(desc(scale=scale)) == sl.LSTM_ERR_INVALID_ARG
    assert decoder.lstm_attn_validate(desc(scale=2.3e38)) == sl.LSTM_OK
    q, k = torch.zeros(2, 3, 4, 64), torch.zeros(2, 5, 2, 64)
    with pytest.raises(ValueError):
        decoder.prepare_attn(q, k, k, scale=1e-60)  # 0 in fp32, which selects 1/sqrt(D)
    with pytest.raises(sl.LstmError):
        decoder.prepare_attn(q, k, k, scale=1e60)


def test_problems_run_on_the_current_device(monkeypatch):
    class Tensor:
        device = torch.device("cuda:1")

    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 64 * index, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    assert decoder._on(None, Tensor) == 64 and decoder._on(7, Tensor) == 7
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    for stream in (None, 7):
        with pytest.raises(ValueError):
            decoder._on(stream, Tensor)
