"""Beam search with an attentional encoder-decoder of stacked LSTMs, all on the library:

    encoder   lstm_fwd over the source, its outputs are k and v (read in place, step by sentence)
    per step  lstm_fwd of one step for every beam, lstm_attn_fwd of the beams of a sentence over its
              encoder outputs, a linear layer, lstm_beam_step (selection, reordering of h and c)

Random weights; prints the best hypothesis of each sentence and the time of a step.

    python examples/beam_decode.py [--batch 16 --beams 5 --source 50 --steps 20 --hidden 512 --layers 2]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import stacked_lstm_forward_amd as sl  # noqa: E402
from stacked_lstm_forward_amd import decoder, runner  # noqa: E402

BOS, EOS = 1, 2


class Stack:
    """A stack of L LSTM layers of width H over B sequences of T steps: weights, outputs, workspace."""

    def __init__(self, L, H, B, T, weights, dtype, device):
        self.desc = sl.make_desc(L, H, H, B, T, "bf16" if dtype == torch.bfloat16 else "f32")
        self.W, self.R, self.b = weights
        self.ws, _ = runner.workspace(self.desc, device)
        self.y = torch.empty((T, B, H), dtype=dtype, device=device)

    def run(self, x, h0, c0, hT, cT):
        sl.check(sl.lstm_fwd(self.desc, x, h0, c0, self.W, self.R, self.b, self.y, hT, cT, self.ws,
                             torch.cuda.current_stream()), "lstm_fwd")
        return self.y


class Model:
    """Weights of the network: `torch.float32` or `torch.bfloat16`, uniform in +-1/sqrt(H) (stacks) and
    normal (embedding, output layer)."""

    def __init__(self, L, H, V, heads, dtype=torch.bfloat16, device="cuda:0", seed=0):
        g = torch.Generator().manual_seed(seed)
        self.L, self.H, self.V, self.heads, self.dtype, self.device = L, H, V, heads, dtype, device

        def uniform(n):
            return ((2 * torch.rand(n, generator=g) - 1) / H ** 0.5).to(dtype).to(device)

        self.encoder, self.decoder = ((uniform(L * 4 * H * H), uniform(L * 4 * H * H), uniform(L * 4 * H))
                                      for _ in range(2))
        self.embedding = torch.randn(V, H, generator=g).to(dtype).to(device)
        self.out = (torch.randn(2 * H, V, generator=g) * (4 / H) ** 0.5).to(dtype).to(device)


class BeamDecoder:
    """Decodes a batch of B sources of up to S steps with K beams; made once, run for any sources."""

    def __init__(self, model, B, S, K, alpha=0.6):
        m = self.model = model
        L, H, V, dev = m.L, m.H, m.V, m.device
        self.B, self.S, self.K = B, S, K
        self.enc = Stack(L, H, B, S, m.encoder, m.dtype, dev)
        self.dec = Stack(L, H, B * K, 1, m.decoder, m.dtype, dev)
        self.kv_len = torch.empty(B, dtype=torch.int32, device=dev)
        keys = self.enc.y.view(S, B, m.heads, -1).transpose(0, 1)
        self.attn = decoder.prepare_attn(self.dec.y.view(B, K, m.heads, -1), keys, keys, kv_len=self.kv_len)
        self.both = torch.empty((B * K, 2 * H), dtype=m.dtype, device=dev)
        self.logits = torch.empty((B, K, V), dtype=m.dtype, device=dev)
        self.beam = decoder.prepare_beam(
            self.logits, torch.empty((B, K), device=dev), torch.empty((B, K), dtype=torch.uint8, device=dev),
            torch.empty((B, K), dtype=torch.int32, device=dev), eos=EOS, alpha=alpha,
            states=(torch.empty((L, B * K, H), dtype=m.dtype, device=dev), torch.empty((L, B * K, H), device=dev)))

    def start(self, source, lengths):
        """source [S, B] tokens, lengths [B]: encodes, and gives every sentence one live beam.  The decoder
        starts from zeros; all that it knows of the source comes through the attention."""
        s = self.beam
        self.kv_len.copy_(lengths)
        self.enc.run(self.model.embedding[source], None, None, None, None)
        s.scores.fill_(-float("inf"))
        s.scores[:, 0] = 0
        for t in (s.finished, s.lengths, *s.states):
            t.zero_()
        self.tokens = torch.full((self.B, self.K), BOS, dtype=torch.int32, device=source.device)

    def step(self):
        """One token for every beam; returns (tokens, parents) [B, K]."""
        m, s, K = self.model, self.beam, self.K
        y = self.dec.run(m.embedding[self.tokens.view(1, -1)], *s.states, *s.states_out)[0]
        s.states, s.states_out = s.states_out, s.states
        self.attn.forward()
        self.both[:, :m.H] = y
        self.both[:, m.H:] = self.attn.o.reshape(self.B * K, m.H)
        torch.mm(self.both, m.out, out=self.logits.view(self.B * K, m.V))
        s.step()
        self.tokens = s.tokens
        s.advance()
        return s.tokens, s.parents

    def decode(self, source, lengths, steps):
        """Hypotheses [B, K, steps], best first, and their scores (summed log-probabilities) [B, K]."""
        self.start(source, lengths)
        made = [tuple(t.clone() for t in self.step()) for _ in range(steps)]
        at = torch.arange(self.K, device=source.device).expand(self.B, self.K)
        out = []
        for tokens, parents in reversed(made):
            out.append(tokens.gather(1, at))
            at = parents.gather(1, at).long()
        return torch.stack(out[::-1], -1), self.beam.scores


def main():
    a = argparse.ArgumentParser()
    for name, n in (("batch", 16), ("beams", 5), ("source", 50), ("steps", 20), ("hidden", 512), ("layers", 2),
                    ("vocabulary", 32000), ("heads", 8)):
        a.add_argument("--" + name, type=int, default=n)
    a = a.parse_args()
    model = Model(a.layers, a.hidden, a.vocabulary, a.heads)
    g = torch.Generator().manual_seed(1)
    source = torch.randint(3, a.vocabulary, (a.source, a.batch), generator=g).cuda()
    lengths = torch.randint(a.source // 2, a.source + 1, (a.batch,), generator=g).int().cuda()
    d = BeamDecoder(model, a.batch, a.source, a.beams)
    tokens, scores = d.decode(source, lengths, a.steps)
    for b in range(min(a.batch, 4)):
        print(f"{float(scores[b, 0]):9.3f}  {tokens[b, 0].tolist()}")
    d.start(source, lengths)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(a.steps):
        d.step()
    end.record()
    torch.cuda.synchronize()
    print(f"{begin.elapsed_time(end) / a.steps * 1000:.0f} us a step of {a.batch} x {a.beams} beams")


if __name__ == "__main__":
    main()
