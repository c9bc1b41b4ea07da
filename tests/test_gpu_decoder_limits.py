"""The decoder operators at the largest sizes they accept."""
import math

import pytest
import torch

from stacked_lstm_forward_amd import decoder

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
MOST = (1 << 31) - 4096


@pytest.fixture(autouse=True)
def _give_memory_back():
    yield
    torch.cuda.empty_cache()


def test_attention_over_the_longest_key_axis():
    """2^31 - 4096 keys, one row (few-rows kernel) and 40 rows: the last key decides, or is left out."""
    S, D = MOST, 8
    k = torch.zeros(1, S, 1, D, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    k[0, S - 1] = 16.0
    v[0, S - 1, 0] = torch.arange(1, D + 1, device=DEV).to(torch.bfloat16)
    z = 16.0 * 16.0 * D / math.sqrt(D)  # 724: the others' exponentials are 0 beside it
    for Tq in (1, 40):
        q = torch.full((1, Tq, 1, D), 16.0, dtype=torch.bfloat16, device=DEV)
        p = decoder.prepare_attn(q, k, v)
        p.forward()
        assert torch.equal(p.o, v[:, -1:].expand_as(p.o))
        # scale, its product with log2 e, z's product, ln 2, its product, the sum: half a step each
        assert float((p.lse.double() - z).abs().max()) <= 6 * 2.0 ** -24 * z
        n = torch.tensor([S - 1], dtype=torch.int32, device=DEV)
        p = decoder.prepare_attn(q, k, v, kv_len=n)
        p.forward()
        assert float(p.o.abs().max()) == 0
        # sums of ones: exact to 2^24 in a lane, rounded where 8 waves, 4 lane groups and 256 parts join
        assert float((p.lse.double() - math.log(S - 1)).abs().max()) <= (8 + 4 + 256 + 2 * math.log(S)) * 2.0 ** -24
