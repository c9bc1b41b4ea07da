"""Attention: rows that a mask or a length leaves without keys."""
import math

import pytest
import torch

from stacked_lstm_forward_amd import decoder

from .test_gpu_decoder import DEV, DT, check, tensors

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
