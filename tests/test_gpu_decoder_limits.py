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


# A launch holds fewer than 2^32 threads along an axis: the cases below have more.


def rows_of_one_key(B, Tq, seed, train=False):
    """q (and dout) [B, Tq, 1, 8], k, v [B, 1, 1, 8] in bf16: with one key o is v and lse is the score."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def make(*shape):
        x = torch.randn(1 << 20, 8, generator=g, device=DEV).to(torch.bfloat16)  # repeated: quick to fill
        n = math.prod(shape) // 8
        return x.repeat((n + (1 << 20) - 1) >> 20, 1)[:n].view(shape)

    return make(B, Tq, 1, 8), make(B, 1, 1, 8), make(B, 1, 1, 8), make(B, Tq, 1, 8) if train else None


def check_one_key(p, q, k, v):
    assert torch.equal(p.o, v.expand_as(p.o))
    for at in range(0, q.shape[0], 1 << 21):  # in pieces: 64-bit copies of all of it are large
        b = slice(at, at + (1 << 21))
        qd, kd = q[b].double(), k[b].double()
        z, most = (qd * kd).sum(-1)[..., 0] / math.sqrt(8), (qd * kd).abs().sum(-1)[..., 0] / math.sqrt(8)
        # eight products summed, then as in the test above
        assert bool(((p.lse[b, 0].double() - z).abs() <= (8 + 6) * 2.0 ** -24 * most).all()), at


@pytest.mark.parametrize("B,Tq", [((1 << 24) + 5, 1), ((1 << 24) + 3, 33)], ids=["few rows", "row tiles"])
def test_attention_of_many_sentences(B, Tq):
    q, k, v, _ = rows_of_one_key(B, Tq, 1)
    p = decoder.prepare_attn(q, k, v)
    p.o.fill_(math.nan)
    p.forward()
    check_one_key(p, q, k, v)


def test_attention_gradients_of_many_rows():
    # 2^28 rows: 2^32 threads of row statistics, 2^24 workgroups of gradients
    B, Tq = (1 << 23) + 8, 32
    q, k, v, do = rows_of_one_key(B, Tq, 2, train=True)
    p = decoder.prepare_attn(q, k, v, train=True)
    for t in (p.o, p.dq, p.dk, p.dv):
        t.fill_(math.nan)
    p.forward()
    p.backward(do)
    check_one_key(p, q, k, v)
    u, w, scale = 2.0 ** -8, 2.0 ** -24, 1 / math.sqrt(8)
    for at in range(0, B, 1 << 20):
        b = slice(at, at + (1 << 20))
        qd, kd, vd, dd = (t[b].double() for t in (q, k, v, do))
        # p is 1 but for its score's and lse's rounding
        rel = w * ((8 + 4 + 2) * scale * (qd * kd).abs().sum(-1, keepdim=True) + 17)
        want, spread = dd.sum(1, keepdim=True), dd.abs().sum(1, keepdim=True)
        bound = u * want.abs() + ((2.0 ** -16 + rel + 40 * w) * dd.abs()).sum(1, keepdim=True)
        assert bool(((p.dv[b].double() - want).abs() <= bound).all()), at
        # dz is the difference of two sums of the same eight products
        dz = 2 * w * 10 * (dd * vd).abs().sum(-1, keepdim=True) * (1 + rel)
        assert bool((p.dq[b].double().abs() <= 1.01 * scale * dz * kd.abs()).all()), at
        assert bool((p.dk[b].double().abs() <= 1.01 * scale * (dz * qd.abs()).sum(1, keepdim=True)).all()), at


def test_beam_states_of_many_rows():
    # 2^25 rows of h and of c, a wave each
    L, B, K, H, V = 32, (1 << 16) + 1, 16, 8, 17
    g = torch.Generator(device=DEV).manual_seed(3)
    logits = torch.randn(B, K, V, generator=g, device=DEV)
    scores = torch.randn(B, K, generator=g, device=DEV)
    fin = torch.zeros(B, K, dtype=torch.uint8, device=DEV)
    lengths = torch.full((B, K), 3, dtype=torch.int32, device=DEV)
    h, c = (torch.randn(L, B * K, H, generator=g, device=DEV) for _ in range(2))
    s = decoder.prepare_beam(logits, scores, fin, lengths, eos=2, states=(h, c))
    s.step()
    row = (s.parents.long() + K * torch.arange(B, device=DEV)[:, None]).view(-1)
    assert int(s.parents.min()) >= 0 and int(s.parents.max()) < K
    for t, out in ((h, s.states_out[0]), (c, s.states_out[1])):
        assert torch.equal(out, t[:, row])
