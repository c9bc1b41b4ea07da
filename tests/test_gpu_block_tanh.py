"""The gated linear recurrence on the GPU: tanh candidates keep their accuracy relative to themselves."""
import math

import pytest
import torch

from stacked_lstm_forward_amd import block

from .block_reference import W, glr, within
from .test_gpu_block import DEV, DT, Make

pytestmark = pytest.mark.gpu

# tanh(u) of bf16 values relative to itself: below 2^-4 by u - u^3/3, whose next term is 2/15 u^4 < 2^-18.9, and 2
# roundings; from there 1 - 2r, r = 1 / (1 + exp(2|u|)): r is off by 4.2 W of at most 1/2 (2 W of the reciprocal, W of
# the sum and half of the exponential's 2.2 W), z by 4.2 W, at 2^-4 67 W of itself, and one rounding: 2^-17.9
TANH = 2.0 ** -17


def every_bf16(least):
    """All bf16 values from `least` to 2^7 and their negatives, in rows of 64."""
    v = torch.arange(1 << 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[(v.double() >= least) & (v.double() <= 128)]
    v = torch.cat((v, -v))
    return v[:v.numel() // 64 * 64].view(-1, 1, 64)


@pytest.mark.parametrize("T", [1, 3, 600])
def test_glr_tanh_of_every_bf16_value(T):
    """A gate that is shut (2^-126 of the state before is left) makes the last state the last candidate, in fp32."""
    last = every_bf16(2.0 ** -100)
    B = last.shape[0]
    u = torch.zeros(B, T, 64, dtype=torch.bfloat16)
    u[:, -1:] = last
    f = torch.full_like(u, -math.inf)
    p = block.prepare_glr(f.to(DEV), u.to(DEV), tanh=True)
    p.forward()
    z = torch.tanh(last[:, 0].double())
    within(p.cT, (z, TANH * z.abs()), "tanh")


@pytest.mark.parametrize("T", [1, 3, 600])
def test_glr_gradients_of_every_bf16_candidate(T):
    """With the gate half open, no state before and d = 1: df = -z / 4, du = (1 - z^2) / 2."""
    first = every_bf16(2.0 ** -100)
    B = first.shape[0]
    u = torch.zeros(B, T, 64, dtype=torch.bfloat16)
    u[:, :1] = first
    f = torch.zeros_like(u)
    dy = torch.zeros(B, T, 64)
    dy[:, 0] = 1.0
    p = block.prepare_glr(f.to(DEV), u.to(DEV), tanh=True, train=True)
    p.forward()
    p.backward(dy.to(DEV))
    x = first[:, 0].double()
    z, e = torch.tanh(x), torch.exp(-2 * x.abs())
    # sigmoid(0) and its complement: 5 W each at the most, three products
    within(p.df[:, 0], (-z / 4, (TANH + 16 * W) * z.abs() / 4), "df")
    # slope 4 r (1 - r): of r's 3 W + E (E = (2 + 2.6 |u|) W) and 4 roundings; 1 - z^2 of a small z: 2 roundings.  From
    # |u| = 43.7 on exp(2|u|) passes 2^126 and its reciprocal, the smallest normal number, may be 0
    slope = 4 * e / (1 + e) ** 2
    within(p.du[:, 0], (slope / 2, ((7 + 2 + 2.6 * x.abs()) + 8) * W * slope + 2.0 ** -124), "du")


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")], ids=str)
@pytest.mark.parametrize("by", [1e-4, 1e-6, 1e-9])
@pytest.mark.parametrize("T", [1, 40, 1300])
def test_glr_small_candidates(T, by, types):
    """tanh(u) is u to some 1e-8 of itself here: the recurrence of tanh candidates is that of linear ones."""
    dtype, grads = types
    m = Make(2, T, "tbh", 12)
    f, u, o = m.seq(40, dtype, 1.5, 2.0), m.seq(40, dtype, by), m.seq(40, dtype)
    dy = m.seq(40, grads)
    p = block.prepare_glr(f, u, o, tanh=True, train=True, grad_dtype=DT[grads])
    p.forward()
    p.backward(dy)
    want = glr(f, u, o, dy=dy)
    most = glr(f, u.abs(), o, dy=dy.abs())  # what each candidate contributes, without cancellation
    # a candidate is off by W (fma), its square's part and u^2 / 3 < 1.1e-7 (|u| < 6 by): 3.1e-7 = 5.2 W of itself
    rel = 6 * W
    for k in ("y", "cT", "do"):
        value, bound = want[k]
        within(getattr(p, k), (value, bound + rel * most[k][0].abs()), k)
    # df = a (1 - a) (c - z) d: of both c and z, and d without cancellation
    a = torch.sigmoid(f.cpu().double())
    c = most["cT"][0].new_zeros(2, 1, 40)
    plain = glr(f, u.abs(), dy=dy.abs())
    c = torch.cat((c, plain["y"][0][:, :-1]), 1)
    d = most["du"][0] / (1 - a)
    value, bound = want["df"]
    within(p.df, (value, bound + rel * a * (1 - a) * d * (c + u.cpu().double().abs())), "df")
    # the slope: in fp32 4 e / (1 + e)^2 with 15 W (e's 3 twice, and 9), in bf16 a rounding; and u^2, 4 W
    value, bound = want["du"]
    within(p.du, (value, bound + 20 * W * most["du"][0]), "du")


@pytest.mark.parametrize("T", [1, 3, 600])
def test_glr_tanh_of_fp32_values(T):
    """(1 - e) / (1 + e): 6 W, and e's 3 W times 2 e / (1 - e^2) < 2 from 1/4 on; the series below less than 6 W; the
    gate that is shut and its product 5 W."""
    g = torch.Generator().manual_seed(T)
    last = torch.cat([torch.randn(50, 1, 64, generator=g) * 10.0 ** k for k in range(-20, 2)])
    u = torch.zeros(last.shape[0], T, 64)
    u[:, -1:] = last
    p = block.prepare_glr(torch.full_like(u, -math.inf).to(DEV), u.to(DEV), tanh=True)
    p.forward()
    z = torch.tanh(last[:, 0].double())
    within(p.cT, (z, 17 * W * z.abs()), "tanh")
