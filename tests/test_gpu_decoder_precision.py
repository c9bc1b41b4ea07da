"""How exact the decoder operators are, against the plain 64-bit forms.

Attention in bf16: p and dz enter their products with 16 bits, not 8.  Bounds, element by element: the
output's own rounding (u = eps / 2 of the type), 2^-16 of p or dz for their two-part products, the fp32
arithmetic (as in ``decoder_reference``); delta takes o with 16 bits too (o and o_rest).

Beam search: the largest logits' exponentials count in 64 bits, the others' share of the sum in fp32 (all
roundings one way, that share is off by 2^-19 of itself).
"""
import math

import pytest
import torch

from stacked_lstm_forward_amd import decoder

from .decoder_reference import attention, beam
from .test_gpu_decoder import DEV, DT, beam_inputs, check_beam, tensors, within

pytestmark = pytest.mark.gpu
U = torch.finfo(torch.bfloat16).eps / 2
P = 2.0 ** -16  # two roundings to bf16, the second of what the first leaves
W = 2.0 ** -24


def bounds(q, k, v, dout):
    """{name: (value, bound)} of bf16 tensors without masks, float64 on the CPU."""
    B, Tq, Hq, D = q.shape
    S, Hkv = k.shape[1:3]
    G, scale = Hq // Hkv, 1 / math.sqrt(D)

    def t(x):
        return x.transpose(-1, -2).contiguous()

    def wide(x):
        return x.cpu().double().transpose(1, 2).repeat_interleave(G, 1).contiguous()

    def narrow(x):
        return x.view(B, Hkv, G, S, D).sum(2).transpose(1, 2)

    qd, kd, vd, dd = q.cpu().double().transpose(1, 2), wide(k), wide(v), dout.cpu().double().transpose(1, 2)
    z = scale * (qd @ t(kd))
    lse = torch.logsumexp(z, -1, keepdim=True)
    p = torch.exp(z - lse)
    # p: scores' sums of D products, scaling, the exponential's argument and result, the sums over S
    rel = W * ((D + 4) * scale * (qd.abs() @ t(kd.abs())).amax(-1, keepdim=True) + 2 * lse.abs() + S + 16)
    o = p @ vd
    e_o = U * o.abs() + (P + rel) * (p @ vd.abs())
    delta, dp = (dd * o).sum(-1, keepdim=True), dd @ t(vd)
    e_delta = (dd.abs() * ((P + W * (D + 2)) * o.abs() + (P + rel) * (p @ vd.abs()))).sum(-1, keepdim=True)
    dz = p * (dp - delta)
    n = W * (G * Tq + S + 8)
    e_dz = p * (W * (D + 2) * (dd.abs() @ t(vd.abs())) + e_delta) + (P + 2 * rel + n) * dz.abs()
    dq, dk, dv = scale * (dz @ kd), narrow(scale * (t(dz) @ qd)), narrow(t(p) @ dd)
    return {"o": (o.transpose(1, 2), e_o.transpose(1, 2)),
            "dq": (dq.transpose(1, 2), (scale * (e_dz @ kd.abs()) + U * dq.abs()).transpose(1, 2)),
            "dk": (dk, narrow(scale * (t(e_dz) @ qd.abs())) + U * dk.abs()),
            "dv": (dv, narrow(t((P + rel + n) * p) @ dd.abs()) + U * dv.abs())}


@pytest.mark.parametrize("shape", [(2, 300, 700, 4, 2, 64), (1, 600, 530, 2, 2, 128), (2, 200, 300, 2, 1, 80),
                                   (1, 150, 900, 2, 2, 200), (2, 5, 400, 4, 2, 128), (3, 1, 900, 4, 4, 64),
                                   (1, 24, 333, 2, 2, 96), (2, 300, 10, 2, 1, 64), (4, 50, 3, 2, 2, 128),
                                   (1, 40, 5000, 1, 1, 64), (2, 600, 2, 1, 1, 32)], ids=str)
def test_products_hold_p_and_dz_in_sixteen_bits(shape):
    q, k, v, do = tensors(*shape, "bf16", seed=21)
    p = decoder.prepare_attn(q, k, v, train=True)
    p.forward()
    p.backward(do)
    for name, want in bounds(q, k, v, do).items():
        within(getattr(p, name), want, name)
    p.o_rest = None  # without it delta is taken from the rounded o, and o is the same
    o = p.o.clone()
    p.o.zero_()
    p.forward()
    p.backward(do)
    assert torch.equal(p.o, o)
    want = attention(q, k, v, None, None, do)
    for name in ("dq", "dk", "dv"):
        within(getattr(p, name), want[name], name)


def test_long_fp32_sums_round_once_a_tile():
    """32768 equal terms just above 1: added one by one, a sum of 2^14 and more loses what is above 1
    (2e-4 of each term).  Tiles of 32 terms that are added then leave half a step each."""
    n, term = 1 << 15, 1.0 + 7 * 2.0 ** -15
    bound = (n / 32 + 32 + 8) * W  # a tile's own terms, the tiles, p and the last factors
    # dv: one key, 8 heads of 4096 rows share it
    q = torch.zeros(1, n // 8, 8, 32, device=DEV)
    k, v = torch.zeros(1, 1, 1, 32, device=DEV), torch.ones(1, 1, 1, 32, device=DEV)
    p = decoder.prepare_attn(q, k, v, train=True)
    p.forward()
    p.backward(torch.full_like(q, term))
    assert float((p.dv.double() / (n * term) - 1).abs().max()) <= bound
    # o: 32768 keys of equal scores, with rows enough that the key axis is not split
    q = torch.zeros(256, 40, 1, 32, device=DEV)
    k = torch.zeros(1, n, 1, 32, device=DEV).expand(256, n, 1, 32)
    v = torch.full((1, n, 1, 32), term, device=DEV).expand(256, n, 1, 32)
    p = decoder.prepare_attn(q, k, v)
    p.forward()
    assert float((p.o.double() / term - 1).abs().max()) <= bound


# ---- beam search ---------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("above", [1.5, 8.0, 12.0, 14.5, 15.75])
def test_beam_log_probability_of_a_late_peak(above, dtype):
    """One logit near the row's end, `above` the largest of those before it."""
    B, K, V = 6, 3, 20000
    logits, scores, fin, lengths, _, _ = beam_inputs(B, K, V, dtype, seed=31, finished=0)
    g = torch.Generator().manual_seed(32)
    x = torch.randn(B, K, V, generator=g).clamp(max=4.0)
    x[..., V - 5] = 4.0 + above + torch.rand(B, K, generator=g) / 8
    logits.copy_(x.to(DT[dtype]))
    scores.copy_(torch.tensor([0.0, -9.0, -8.0]))
    s = decoder.prepare_beam(logits, scores, fin, lengths, eos=2, alpha=0.0)
    s.step()
    want = beam(logits, scores, fin, lengths, 2, 0.0)[0]["scores"][:, 0]
    got = s.scores_out.cpu().double()[:, 0]
    assert s.tokens[:, 0].tolist() == [V - 5] * B and bool((got <= 0).all())
    rest = -torch.expm1(want)  # the other logits' share of the sum
    assert bool(((got - want).abs() <= 2.0 ** -19 * rest + 2.0 ** -24 * want.abs() + 1e-13).all())


def near_ties(dtype):
    """Every beam's best proposal ranks the same but for the rounding of its score, some 1e-8."""
    B, K, V = 32, 4, 3000
    logits, scores, fin, lengths, h, c = (t.cpu() for t in beam_inputs(B, K, V, dtype, seed=33, finished=0))
    g = torch.Generator().manual_seed(34)
    x = torch.randn(B, K, V, generator=g) - 70.0
    at = torch.rand(B, K, V, generator=g).argsort(-1)[..., :3]
    x.scatter_(-1, at, torch.rand(B, K, 3, generator=g) * torch.tensor([1.0, 1.0, 0.0]) + torch.tensor([0.0, 0.0, 2.0]))
    logits.copy_(x.to(DT[dtype]))
    d = logits.double()
    scores.copy_((torch.logsumexp(d, -1) - d.amax(-1) - 0.01).float())
    lengths.fill_(7)
    return logits, scores, fin, lengths, h, c


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_beam_proposals_closer_than_fp32_tells_apart(dtype):
    # three logits hold all of each sum: the log-sum-exp is as exact as 64 bits
    check_beam(*(t.to(DEV) for t in near_ties(dtype)), gap=1e-13)
