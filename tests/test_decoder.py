"""CPU tests of the decoder operators: exports, sizes and refusals (host checks; nothing is launched)."""
import os
import re

import pytest
import torch

import stacked_lstm_forward_amd as sl
from stacked_lstm_forward_amd import decoder

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # an aligned address that is never read


def desc(B=2, Tq=3, S=5, Hq=4, Hkv=2, D=64, dtype="bf16", **over):
    s = {n: decoder.AttnStride(t * heads * D, heads * D, D)
         for n, t, heads in (("q", Tq, Hq), ("o", Tq, Hq), ("dout", Tq, Hq), ("dq", Tq, Hq), ("k", S, Hkv),
                             ("v", S, Hkv), ("dk", S, Hkv), ("dv", S, Hkv))}
    d = decoder.AttnDesc(B, Tq, S, Hq, Hkv, D, {"f32": sl.LSTM_F32, "bf16": sl.LSTM_BF16}.get(dtype, dtype), 0.0)
    for n, x in s.items():
        setattr(d, n, x)
    for n, x in over.items():
        setattr(d, n, x)
    return d


def test_every_declared_symbol_is_exported():
    text = open(os.path.join(ROOT, "include", "decoder", "lstm_dec.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^(?:lstm_status_t|size_t)\s+([a-z_]+)\(", text, re.M)
    assert set(names) == set(decoder.EXPORTED)
    for n in names:
        assert hasattr(sl.load_library(), n)


@pytest.mark.parametrize("change,status", [
    (dict(B=0), sl.LSTM_ERR_INVALID_ARG), (dict(Tq=0), sl.LSTM_ERR_INVALID_ARG), (dict(S=-1), sl.LSTM_ERR_INVALID_ARG),
    (dict(Hq=3), sl.LSTM_ERR_INVALID_ARG), (dict(Hkv=0), sl.LSTM_ERR_INVALID_ARG), (dict(dtype=7), sl.LSTM_ERR_INVALID_ARG),
    (dict(scale=-1.0), sl.LSTM_ERR_INVALID_ARG), (dict(scale=float("nan")), sl.LSTM_ERR_INVALID_ARG),
    (dict(scale=float("inf")), sl.LSTM_ERR_INVALID_ARG),
    (dict(D=12), sl.LSTM_ERR_UNSUPPORTED), (dict(D=264), sl.LSTM_ERR_UNSUPPORTED),
    (dict(q=decoder.AttnStride(4, 64, 64)), sl.LSTM_ERR_UNSUPPORTED),
    (dict(k=decoder.AttnStride(640, 64, 65)), sl.LSTM_ERR_UNSUPPORTED),
    (dict(B=1 << 16, S=1 << 16), sl.LSTM_ERR_UNSUPPORTED), (dict(B=1 << 20, Tq=1 << 10), sl.LSTM_ERR_UNSUPPORTED),
    (dict(S=0), sl.LSTM_OK), (dict(D=8), sl.LSTM_OK), (dict(D=200), sl.LSTM_OK), (dict(Hq=128, Hkv=1), sl.LSTM_OK),
])
def test_attention_descriptions(change, status):
    d = desc(**{k: v for k, v in change.items() if k in ("B", "Tq", "S", "D", "dtype", "Hq", "Hkv")})
    for k, v in change.items():
        setattr(d, k, v)
    assert decoder.lstm_attn_validate(d) == status
    assert (decoder.lstm_attn_workspace_size(d) > 0) == (status == sl.LSTM_OK)
    args = [FAKE] * 3 + [None, None] + [FAKE] * 3
    if status != sl.LSTM_OK:
        assert decoder.lstm_attn_fwd(d, *args, stream=0) == status


def test_attention_refuses_pointers():
    d = desc()
    ok = [FAKE, FAKE, FAKE, None, None, FAKE, FAKE, FAKE]
    for i in (0, 1, 2, 5):  # q, k, v, o
        assert decoder.lstm_attn_fwd(d, *[None if j == i else x for j, x in enumerate(ok)], stream=0) == \
            sl.LSTM_ERR_INVALID_ARG
        assert decoder.lstm_attn_fwd(d, *[FAKE + 8 if j == i else x for j, x in enumerate(ok)], stream=0) == \
            sl.LSTM_ERR_UNSUPPORTED
    for ws in (None, FAKE + 16):
        assert decoder.lstm_attn_fwd(d, *ok[:-1], ws, stream=0) == sl.LSTM_ERR_WORKSPACE
    assert decoder.lstm_attn_fwd(None, *ok, stream=0) == sl.LSTM_ERR_INVALID_ARG
    ok = [FAKE, FAKE, FAKE, None, None] + [FAKE] * 7
    for i in (0, 1, 2, 5, 6, 7, 8, 9, 10):
        assert decoder.lstm_attn_bwd(d, *[None if j == i else x for j, x in enumerate(ok)], stream=0) == \
            sl.LSTM_ERR_INVALID_ARG
    assert decoder.lstm_attn_bwd(d, *ok[:-1], FAKE + 4, stream=0) == sl.LSTM_ERR_WORKSPACE
    bad = desc(dk=decoder.AttnStride(640, 4, 64))
    assert decoder.lstm_attn_validate(bad) == sl.LSTM_OK
    assert decoder.lstm_attn_validate(bad, train=True) == sl.LSTM_ERR_UNSUPPORTED
    assert decoder.lstm_attn_bwd(bad, *ok, stream=0) == sl.LSTM_ERR_UNSUPPORTED


def test_prepare_attn_refuses():
    q, k = torch.zeros(2, 3, 4, 64), torch.zeros(2, 5, 2, 64)
    for bad in ((q[0], k, k), (q, k, k[:, :4]), (q, k[:1], k[:1]), (q, torch.zeros(2, 5, 2, 32), k)):
        with pytest.raises(ValueError):
            decoder.prepare_attn(*bad)
    with pytest.raises(TypeError):
        decoder.prepare_attn(q.half(), k.half(), k.half())
    with pytest.raises(TypeError):
        decoder.prepare_attn(q, k.bfloat16(), k)
    with pytest.raises(ValueError):  # the values of a head are not contiguous
        decoder.prepare_attn(q, k.transpose(2, 3).contiguous().transpose(2, 3), k)
    with pytest.raises(ValueError):  # misaligned
        decoder.prepare_attn(torch.zeros(2 * 3 * 4 * 64 + 1)[1:].view(2, 3, 4, 64), k, k)
    with pytest.raises(TypeError):
        decoder.prepare_attn(q, k, k, kv_len=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        decoder.prepare_attn(q, k, k, kv_len=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        decoder.prepare_attn(q, k, k, key_mask=torch.zeros(2, 5))
    with pytest.raises(ValueError):
        decoder.prepare_attn(q, k, k, key_mask=torch.zeros(2, 6, dtype=torch.bool))
    with pytest.raises(ValueError):
        decoder.prepare_attn(q, k, k, scale=0.0)
    with pytest.raises(sl.LstmError):
        decoder.prepare_attn(torch.zeros(2, 3, 3, 64), k, k)
    p = decoder.prepare_attn(q, k, k)
    with pytest.raises(RuntimeError):
        p.backward(torch.zeros_like(q))
    p = decoder.prepare_attn(q, k, k, train=True)
    with pytest.raises(ValueError):
        p.backward(torch.zeros(2, 3, 4, 32))
    assert p.o.shape == q.shape and p.lse.shape == (2, 4, 3) and p.dk.shape == k.shape


def test_outputs_take_the_inputs_layout():
    q = torch.zeros(3, 2, 4, 64).transpose(0, 1)  # [T][B] storage
    p = decoder.prepare_attn(q, q, q, train=True)
    assert p.o.stride() == q.stride() == p.dk.stride()


def test_beam_descriptions():
    good = dict(B=2, K=4, V=100, dtype=sl.LSTM_F32, eos=2, alpha=0.6, L=1, H=8, logits_stride=0)

    def size(**over):
        return decoder.lstm_beam_workspace_size(decoder.BeamDesc(**{**good, **over}))

    assert size() > 0 and size(K=16) > 0 and size(V=1 << 20) > 0 and size(L=0, H=0) > 0 and size(K=1, V=3) > 0
    for over in (dict(B=0), dict(K=0), dict(V=0), dict(K=17), dict(K=4, V=3), dict(dtype=5), dict(eos=-1), dict(eos=100),
                 dict(alpha=-0.1), dict(alpha=float("nan")), dict(L=1, H=0), dict(L=0, H=8), dict(logits_stride=99),
                 dict(V=(1 << 20) + 1), dict(B=1 << 23), dict(L=1 << 12, H=1 << 12)):
        assert size(**over) == 0, over
    d = decoder.BeamDesc(**good)
    ok = [FAKE] * 14
    for i in range(9):
        args = [None if j == i else x for j, x in enumerate(ok)]
        assert decoder.lstm_beam_step(d, *args, stream=0) == sl.LSTM_ERR_INVALID_ARG
    for i, ws in ((11, FAKE), (12, FAKE)):  # a state without its output
        args = [None if j == i else x for j, x in enumerate(ok)]
        assert decoder.lstm_beam_step(d, *args, stream=0) == sl.LSTM_ERR_INVALID_ARG
    assert decoder.lstm_beam_step(d, *ok[:-1], FAKE + 8, stream=0) == sl.LSTM_ERR_WORKSPACE
    assert decoder.lstm_beam_step(d, FAKE + 2, *ok[1:], stream=0) == sl.LSTM_ERR_INVALID_ARG
    assert decoder.lstm_beam_step(None, *ok, stream=0) == sl.LSTM_ERR_INVALID_ARG


def test_prepare_beam_refuses():
    x, s = torch.zeros(2, 4, 50), torch.zeros(2, 4)
    f, n = torch.zeros(2, 4, dtype=torch.uint8), torch.zeros(2, 4, dtype=torch.int32)
    for bad in ((x[0], s, f, n), (x, s[:1], f, n), (x.transpose(1, 2).contiguous().transpose(1, 2), s, f, n)):
        with pytest.raises(ValueError):
            decoder.prepare_beam(*bad, eos=2)
    for bad in ((x.half(), s, f, n), (x, s.double(), f, n), (x, s, f.float(), n), (x, s, f, n.long())):
        with pytest.raises(TypeError):
            decoder.prepare_beam(*bad, eos=2)
    with pytest.raises(ValueError):
        decoder.prepare_beam(x, s, f, n, eos=50)
    with pytest.raises(ValueError):
        decoder.prepare_beam(x, s, f, n, eos=2, states=(torch.zeros(1, 7, 8), None))
    with pytest.raises(TypeError):
        decoder.prepare_beam(x, s, f, n, eos=2, states=(None, torch.zeros(1, 8, 8).bfloat16()))
    p = decoder.prepare_beam(x, s, f.bool(), n, eos=2, states=(torch.zeros(1, 8, 8), torch.zeros(1, 8, 8)))
    assert p.tokens.shape == (2, 4) and p.states_out[0].shape == (1, 8, 8)
    before = p.scores_out
    p.advance()
    assert p.scores is before


def test_the_plain_forms():
    """The references used on the GPU, against torch's autograd and a brute force over proposals."""
    from .decoder_reference import attention, beam
    g = torch.Generator().manual_seed(0)
    q, k, v, do = (torch.randn(2, n, h, 8, generator=g, dtype=torch.float64)
                   for n, h in ((3, 4), (5, 2), (5, 2), (3, 4)))
    n = torch.tensor([4, 5], dtype=torch.int32)
    ref = attention(q, k, v, n, None, do)
    qq, kk, vv = (x.clone().requires_grad_() for x in (q, k, v))
    z = torch.einsum("bthd,bshd->bhts", qq, kk.repeat_interleave(2, 2)) / 8 ** 0.5
    z = z.masked_fill(torch.arange(5)[None, None, None] >= n[:, None, None, None], -float("inf"))
    o = torch.einsum("bhts,bshd->bthd", z.softmax(-1), vv.repeat_interleave(2, 2))
    (o * do).sum().backward()
    for name, x in (("o", o), ("dq", qq.grad), ("dk", kk.grad), ("dv", vv.grad)):
        assert torch.allclose(ref[name][0], x, atol=1e-12), name
    logits = torch.randn(1, 2, 4, generator=g)
    scores = torch.tensor([[-1.0, -0.5]])
    fin, lens = torch.tensor([[0, 1]], dtype=torch.uint8), torch.tensor([[2, 3]], dtype=torch.int32)
    got, _ = beam(logits, scores, fin, lens, 1, 0.6)
    every = [((scores[0, 0].double() + logits[0, 0].double().log_softmax(-1)[t]) / (8 / 6) ** 0.6, 0, t) for t in range(4)]
    every.append((scores[0, 1].double() / (8 / 6) ** 0.6, 1, 1))
    every.sort(key=lambda x: (-float(x[0]), x[1], x[2]))
    assert [(x[1], x[2]) for x in every[:2]] == list(zip(got["parents"][0].tolist(), got["tokens"][0].tolist()))
