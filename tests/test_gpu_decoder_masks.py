"""Attention: rows without keys, the few-rows kernel's instances with and without masks, large scores."""
import math

import pytest
import torch

from stacked_lstm_forward_amd import decoder

from .decoder_reference import attention
from .test_gpu_decoder import DEV, DT, check, tensors, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(3, 3, 200, 4, 2, 64), (3, 24, 90, 2, 2, 96), (3, 90, 300, 2, 1, 64),
                                   (3, 300, 600, 4, 2, 128), (3, 1, 5000, 2, 2, 64), (3, 40, 700, 1, 1, 200)], ids=str)
def test_rows_without_keys_whatever_q_and_dout_hold(shape, dtype):
    q, k, v, do = tensors(*shape, dtype, seed=41)
    m = torch.rand(shape[0], shape[2], generator=torch.Generator().manual_seed(42)) < 0.7
    m[1] = False  # left without keys by the mask, sentence 2 by its length
    n = torch.tensor([shape[2], shape[2], 0], dtype=torch.int32)
    bad = torch.tensor([math.nan, math.inf, -math.inf, 1.0, 0.0]).to(DT[dtype]).to(DEV)
    for t in (q, do):
        for b in (1, 2):
            t[b] = bad[torch.arange(t[b].numel(), device=DEV) % 5].view(t[b].shape)
    p = decoder.prepare_attn(q, k, v, kv_len=n.to(DEV), key_mask=m.to(DEV), train=True)
    for t in (p.o, p.lse, p.dq, p.dk, p.dv):
        t.fill_(math.nan)
    p.forward()
    p.backward(do)
    for b in (1, 2):
        assert bool((p.lse[b] == -math.inf).all())
        for name in ("o", "dq", "dk", "dv"):
            assert bool((getattr(p, name)[b] == 0).all()), (b, name)
    check(q[:1], k[:1], v[:1], do[:1], key_mask=m[:1].to(DEV))  # the sentence with keys
    assert bool(torch.isfinite(p.o[0]).all()) and bool(torch.isfinite(p.dq[0]).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [(1, 3), (10, 2)], ids=["one group of rows", "two groups"])
@pytest.mark.parametrize("S", [50, 700], ids=["few keys", "many keys"])
@pytest.mark.parametrize("D", [24, 96, 128, 152, 160, 192, 200, 224, 248])
def test_few_rows(D, S, rows, dtype):
    Tq, G = rows
    q, k, v, do = tensors(3, Tq, S, 2 * G, 2, D, dtype, seed=43)
    m = torch.rand(3, S, generator=torch.Generator().manual_seed(44)) < 0.6
    m[1, : S // 2] = False
    n = torch.tensor([S, S - 3, S // 2], dtype=torch.int32)
    check(q, k, v, do, train=False)
    bad = torch.tensor([math.nan, math.inf, -math.inf])[torch.arange(S) % 3].to(DT[dtype])
    for x in (k, v):  # what the mask leaves out is never used
        x.copy_(torch.where(m[:, :, None, None], x.cpu(), bad[None, :, None, None]))
    check(q, k, v, do, key_mask=m.to(DEV), train=False)
    check(q, k, v, do, kv_len=n.to(DEV), key_mask=m.to(DEV), train=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("by", [30.0, 300.0])
def test_gradients_of_large_scores(by, dtype):
    # p is taken from scores and lse of some 100 to 1000, in fp32, where it underflows below 2^-126: added
    # to the reference's bounds, with the largest that p and dz are multiplied by and summed over
    for shape, seed in (((2, 18, 260, 2, 2, 32), 5), ((1, 70, 600, 4, 2, 64), 45)):
        q, k, v, do = tensors(*shape, dtype, seed=seed, q_by=by)
        p = decoder.prepare_attn(q, k, v, train=True)
        p.forward()
        p.backward(do)
        qm, km, vm, dm = (float(t.abs().max()) for t in (q, k, v, do))
        B, Tq, S, Hq, Hkv, D = shape
        rows = Tq * (Hq // Hkv)
        dz = 1 + 2 * D * dm * vm  # |dP - delta|, and a rounding of dz itself
        most = {"o": S * vm, "dv": rows * dm, "dk": rows * dz * qm, "dq": S * dz * km}
        for name, (value, bound) in attention(q, k, v, None, None, do).items():
            within(getattr(p, name), (value, bound + 2.0 ** -126 * (1 + most.get(name, 0.0))), name)
