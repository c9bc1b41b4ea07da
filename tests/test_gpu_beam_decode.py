"""Beam search of an encoder-decoder through the stacks, the attention and the beam step together."""
import math
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def stack(x, W, R, b, L, H):
    """The LSTM stack in float64: x [T, B, H] -> y [T, B, H]."""
    W, R, b = W.double().view(L, 4 * H, H), R.double().view(L, 4 * H, H), b.double().view(L, 4 * H)
    for l in range(L):
        h = c = torch.zeros(x.shape[1], H, dtype=torch.float64)
        out = []
        for u in x:
            i, f, g, o = (u @ W[l].t() + h @ R[l].t() + b[l]).chunk(4, -1)
            c = f.sigmoid() * c + i.sigmoid() * g.tanh()
            h = o.sigmoid() * c.tanh()
            out.append(h)
        x = torch.stack(out)
    return x


def test_beam_decode_scores_are_the_models():
    import beam_decode as bd
    L, H, V, heads, B, S, K, steps = 2, 64, 101, 2, 3, 9, 4, 6
    m = bd.Model(L, H, V, heads, torch.float32)
    g = torch.Generator().manual_seed(5)
    source = torch.randint(3, V, (S, B), generator=g)
    lengths = torch.tensor([9, 1, 5], dtype=torch.int32)
    d = bd.BeamDecoder(m, B, S, K)
    tokens, scores = d.decode(source.cuda(), lengths.cuda(), steps)
    again, _ = d.decode(source.cuda(), lengths.cuda(), steps)  # made once, run again
    assert torch.equal(tokens, again)
    tokens, scores = tokens.cpu().long(), scores.cpu().double()
    # each hypothesis teacher-forced through the network in 64 bits
    emb, out = m.embedding.cpu().double(), m.out.cpu().double()
    enc = stack(emb[source], *(w.cpu() for w in m.encoder), L, H).view(S, B, heads, -1)
    previous = torch.cat([torch.full((B, K, 1), bd.BOS), tokens[..., :-1]], -1)
    y = stack(emb[previous.view(B * K, steps).t()], *(w.cpu() for w in m.decoder), L, H).view(steps, B, K, heads, -1)
    total = torch.zeros(B, K, dtype=torch.float64)
    for b in range(B):
        e = enc[:lengths[b], b]
        p = (torch.einsum("tkhd,shd->tkhs", y[:, b], e) / math.sqrt(H // heads)).softmax(-1)
        ctx = torch.einsum("tkhs,shd->tkhd", p, e)
        lp = (torch.cat([y[:, b].flatten(2), ctx.flatten(2)], -1) @ out).log_softmax(-1)
        for k in range(K):
            for t in range(steps):
                total[b, k] += lp[t, k, tokens[b, k, t]]
                if tokens[b, k, t] == bd.EOS:
                    assert bool((tokens[b, k, t:] == bd.EOS).all())
                    break
    # fp32 products of up to 128 terms in each of six steps, logits of size 10: some 1e-5 a step
    assert float((scores - total).abs().max()) < 6 * 1e-4
    assert len({tuple(x) for x in tokens[0].tolist()}) == K  # no hypothesis twice
