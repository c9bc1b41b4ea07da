"""How exact the attention's 16-bit products are: p and dz enter them with 16 bits, not 8.

Bounds against the plain 64-bit forms, element by element: the output's own rounding (u = eps / 2 of the
type), 2^-16 of p or dz for their two-part products, the fp32 arithmetic (as in ``decoder_reference``),
and for dq and dk the rounding of the o that delta is taken from.
"""
import math

import pytest
import torch

from stacked_lstm_forward_amd import decoder

from .test_gpu_decoder import tensors, within

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
    e_delta = (dd.abs() * (e_o + W * (D + 2) * o.abs())).sum(-1, keepdim=True)
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
                                   (1, 24, 333, 2, 2, 96)], ids=str)
def test_products_hold_p_and_dz_in_sixteen_bits(shape):
    q, k, v, do = tensors(*shape, "bf16", seed=21)
    p = decoder.prepare_attn(q, k, v, train=True)
    p.forward()
    p.backward(do)
    for name, want in bounds(q, k, v, do).items():
        within(getattr(p, name), want, name)
