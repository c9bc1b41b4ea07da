"""The decoder operators on the GPU against their plain 64-bit forms."""
import math

import pytest
import torch

from stacked_lstm_forward_amd import decoder

from .decoder_reference import attention, beam

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def tensors(B, Tq, S, Hq, Hkv, D, dtype, layout="tbh", seed=0, q_by=1.5):
    g = torch.Generator().manual_seed(seed)

    def make(T, heads, by=1.0):
        if layout == "tbh":
            x = torch.randn(T, B, heads, D, generator=g).mul_(by).to(DT[dtype]).to(DEV)
            return x.transpose(0, 1)
        if layout == "bht":
            x = torch.randn(B, heads, T, D, generator=g).mul_(by).to(DT[dtype]).to(DEV)
            return x.transpose(1, 2)
        if layout == "wide":  # a slice of a wider tensor: every stride larger than dense
            x = torch.randn(B, T, heads + 1, D + 16, generator=g).mul_(by).to(DT[dtype]).to(DEV)
            return x[:, :, 1:, 8:D + 8]
        return torch.randn(B, T, heads, D, generator=g).mul_(by).to(DT[dtype]).to(DEV)

    return make(Tq, Hq, q_by), make(S, Hkv), make(S, Hkv), make(Tq, Hq)


def within(got, want, what):
    value, bound = want
    got = got.cpu().double()
    assert got.shape == value.shape, what
    inf = torch.isinf(value)
    assert torch.equal(got[inf], value[inf]), f"{what}: infinities"
    d = (got - value).abs()[~inf]
    ok = d <= bound[~inf]  # false for NaN
    assert bool(ok.all()), f"{what}: off by {float((d / bound[~inf].clamp(min=1e-300)).max()):.3g} of the bound"


def check(q, k, v, dout, kv_len=None, key_mask=None, train=True, scale=None):
    p = decoder.prepare_attn(q, k, v, kv_len=kv_len, key_mask=key_mask, train=train, scale=scale)
    for t in (p.o, p.lse, p.dq, p.dk, p.dv):
        if t is not None:
            t.fill_(math.nan)  # every element is written
    p.forward()
    want = attention(q, k, v, kv_len, key_mask, dout if train else None, scale)
    names = ["o", "lse"]
    if train:
        p.backward(dout)
        names += ["dq", "dk", "dv"]
    for n in names:
        within(getattr(p, n), want[n], n)
    return p


SHAPES = [
    # B, Tq, S, Hq, Hkv, D
    (1, 1, 1, 1, 1, 8),
    (2, 3, 5, 2, 1, 32),
    (3, 16, 64, 2, 2, 64),
    (2, 17, 65, 4, 2, 80),
    (1, 130, 129, 1, 1, 96),
    (2, 33, 200, 6, 2, 128),
    (1, 65, 31, 3, 1, 136),
    (1, 40, 100, 2, 2, 192),
    (1, 20, 90, 2, 1, 200),
    (2, 70, 140, 2, 2, 256),
    (1, 300, 1100, 2, 1, 64),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_attention(shape, dtype):
    q, k, v, do = tensors(*shape, dtype)
    check(q, k, v, do)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(3, 300, 600, 4, 2, 24), (3, 270, 550, 4, 2, 64), (3, 530, 560, 1, 1, 80),
                                   (3, 180, 600, 9, 3, 128), (3, 600, 520, 1, 1, 160)], ids=str)
def test_attention_of_many_rows_and_keys(shape, dtype):
    B, Tq, S = shape[:3]
    q, k, v, do = tensors(*shape, dtype, seed=14)
    n = torch.tensor([S, 0, S // 2 + 5], dtype=torch.int32)
    m = torch.rand(B, S, generator=torch.Generator().manual_seed(15)) < 0.7
    bad = torch.tensor([math.nan, math.inf, -math.inf])[torch.arange(S) % 3].to(DT[dtype])
    check(q, k, v, do)
    for x in (k, v):  # what the mask leaves out is never used
        x.copy_(torch.where(m[:, :, None, None], x.cpu(), bad[None, :, None, None]))
    check(q, k, v, do, kv_len=n.to(DEV), key_mask=m.to(DEV))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["bth", "bht", "wide"])
def test_attention_layouts(layout, dtype):
    q, k, v, do = tensors(2, 21, 77, 4, 2, 64, dtype, layout, seed=1)
    check(q, k, v, do)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(5, 19, 90, 4, 2, 64), (5, 1, 700, 8, 2, 128), (5, 150, 333, 2, 2, 80)], ids=str)
def test_attention_masks(shape, dtype):
    B, Tq, S = shape[:3]
    q, k, v, do = tensors(*shape, dtype, seed=2)
    g = torch.Generator().manual_seed(3)
    n = torch.tensor([S, 0, 1, S // 2 + 1, -4], dtype=torch.int32)
    m = torch.rand(B, S, generator=g) < 0.6
    m[3] = False  # a row that the mask empties
    m[0, : S // 2] = False
    check(q, k, v, do, kv_len=n.to(DEV))
    check(q, k, v, do, key_mask=m.to(DEV))
    check(q, k, v, do, kv_len=(n + 3).to(DEV), key_mask=m.to(torch.uint8).to(DEV))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Tq", [1, 40])
def test_attention_ignores_what_is_masked(Tq, dtype):
    q, k, v, do = tensors(3, Tq, 150, 4, 2, 64, dtype, seed=4)
    n = torch.tensor([150, 70, 0], dtype=torch.int32)
    m = torch.ones(3, 150, dtype=torch.uint8)
    m[0, 3:140:7] = 0
    keep = (torch.arange(150)[None] < n[:, None]) & m.bool()
    bad = torch.tensor([math.nan, math.inf, -math.inf])[torch.arange(150) % 3].to(DT[dtype])
    for x in (k, v):
        x.copy_(torch.where(keep[:, :, None, None], x.cpu(), bad[None, :, None, None]))
    check(q, k, v, do, kv_len=n.to(DEV), key_mask=m.to(DEV))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_without_keys(dtype):
    q, k, v, do = tensors(2, 9, 0, 2, 1, 64, dtype)
    p = check(q, k, v, do)
    assert float(p.o.abs().max()) == 0 and bool((p.lse == -math.inf).all()) and float(p.dq.abs().max()) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("by", [30.0, 300.0])
def test_attention_of_large_scores(by, dtype):
    # one key decides: the running maximum moves by far more than the exponent's range
    q, k, v, do = tensors(2, 18, 260, 2, 2, 32, dtype, seed=5, q_by=by)
    p = decoder.prepare_attn(q, k, v, train=True)
    p.forward()
    p.backward(do)
    want = attention(q, k, v, dout=do)
    within(p.o, want["o"], "o")
    within(p.lse, want["lse"], "lse")
    for t in (p.dq, p.dk, p.dv):
        assert bool(torch.isfinite(t).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 5000, 8, 8, 64), (2, 5, 3001, 8, 2, 128), (1, 8, 2500, 16, 2, 64),
                                   (3, 2, 900, 5, 1, 256), (1, 1, 20, 1, 1, 80)], ids=str)
def test_attention_single_steps(shape, dtype):
    q, k, v, do = tensors(*shape, dtype, "bth", seed=6)
    n = torch.full((shape[0],), shape[2] - 3, dtype=torch.int32, device=DEV)
    check(q, k, v, do, train=False)
    check(q, k, v, do, kv_len=n, train=False)


def test_attention_scale_and_no_lse():
    q, k, v, do = tensors(2, 11, 50, 2, 2, 64, "f32", seed=7)
    check(q, k, v, do, scale=0.3)
    p = decoder.prepare_attn(q, k, v)
    p.forward()
    o = p.o.clone()
    p.lse = None
    p.o.zero_()
    p.forward()
    assert torch.equal(o, p.o)


def test_attention_gradient_against_differences():
    q, k, v, do = tensors(1, 6, 9, 2, 1, 32, "f32", seed=8)
    n = torch.tensor([8], dtype=torch.int32)
    p = decoder.prepare_attn(q, k, v, kv_len=n.to(DEV), train=True)
    p.forward()
    p.backward(do)
    g = torch.Generator().manual_seed(9)
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        r = torch.randn(x.shape, generator=g).double()
        step = 2.0 ** -10

        def loss(sign):
            args = {"q": q.cpu().double(), "k": k.cpu().double(), "v": v.cpu().double()}
            args[name[1]] = args[name[1]] + sign * step * r
            return (attention(args["q"], args["k"], args["v"], n)["o"][0] * do.cpu().double()).sum()

        slope = float((loss(1) - loss(-1)) / (2 * step))
        # central differences: off by step^2 / 6 of the third derivative, about 1e-6 of the terms' sum
        got = getattr(p, name).cpu().double() * r
        assert abs(float(got.sum()) - slope) <= 1e-4 * float(got.abs().sum())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_is_deterministic_and_captures(dtype):
    q, k, v, do = tensors(3, 60, 500, 4, 2, 64, dtype, seed=10)
    n = torch.tensor([500, 0, 333], dtype=torch.int32, device=DEV)
    p = decoder.prepare_attn(q, k, v, kv_len=n, train=True)
    one = decoder.prepare_attn(q[:, :1], k, v, kv_len=n)
    names = ("o", "lse", "dq", "dk", "dv")

    def step():
        p.forward()
        p.backward(do)
        one.forward()

    step()
    first = [getattr(p, x).clone() for x in names] + [one.o.clone(), one.lse.clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    again = [getattr(p, x) for x in names] + [one.o, one.lse]
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        q.mul_(-1.0)  # new inputs between the replays
        step()
        first = [x.clone() for x in again]
        for x in again:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again)), i


def test_attention_far_offsets():
    # the last sentence's keys start beyond 2^31 elements
    B, S, D = 2, 64, 64
    far = (1 << 31) + (1 << 20)
    buf = torch.empty(far + S * D, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(11)
    kv = torch.randn(B, S, D, generator=g).to(torch.bfloat16).to(DEV)
    k = torch.as_strided(buf, (B, S, 1, D), (far, D, D, 1))
    k.copy_(kv[:, :, None])
    q, _, v, do = tensors(B, 20, S, 1, 1, D, "bf16", "bth", seed=12)
    p = decoder.prepare_attn(q, k, v)
    p.forward()
    want = attention(q, k, v)
    within(p.o, want["o"], "o")
    within(p.lse, want["lse"], "lse")


# ---- beam search ---------------------------------------------------------------


def beam_inputs(B, K, V, dtype, seed=0, H=8, L=2, finished=0.2):
    g = torch.Generator().manual_seed(seed)
    logits = (2.5 * torch.randn(B, K, V, generator=g)).to(DT[dtype])
    if V > 1:
        logits[..., 0] = -math.inf
    lengths = torch.randint(1, 30, (B, K), generator=g, dtype=torch.int32)
    scores = -lengths * (0.2 + torch.rand(B, K, generator=g))
    fin = (torch.rand(B, K, generator=g) < finished).to(torch.uint8)
    h = torch.randn(L, B * K, H, generator=g).to(DT[dtype])
    c = torch.randn(L, B * K, H, generator=g)
    return [x.to(DEV) for x in (logits, scores, fin, lengths, h, c)]


def check_beam(logits, scores, fin, lengths, h=None, c=None, eos=2, alpha=0.6, gap=1e-6):
    B, K, V = logits.shape
    s = decoder.prepare_beam(logits, scores, fin, lengths, eos=eos, alpha=alpha, states=(h, c))
    s.step()
    want, least = beam(logits, scores, fin, lengths, eos, alpha)
    assert least > gap  # of the inputs: ranks closer than the logits' exponentials allow are not tested here
    for name, got in (("tokens", s.tokens), ("parents", s.parents), ("finished", s.finished_out),
                      ("lengths", s.lengths_out)):
        assert torch.equal(got.cpu(), want[name]), name
    # exponentials within 2 steps of fp32 (2^-22), the score's own rounding
    got, ref = s.scores_out.cpu().double(), want["scores"]
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf])
    assert bool(((got - ref).abs() <= 2.0 ** -22 + 2.0 ** -24 * ref.abs())[~inf].all())
    row = (want["parents"].long() + K * torch.arange(B)[:, None]).view(-1)
    for t, out in ((h, s.states_out[0]), (c, s.states_out[1])):
        if t is not None:
            assert torch.equal(out.cpu(), t.cpu()[:, row])
    return s


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 3), (2, 4, 5), (3, 5, 1001), (2, 16, 4099), (5, 8, 32007), (1, 3, 150001),
                                   (40, 2, 515)], ids=str)
def test_beam(shape, dtype):
    check_beam(*beam_inputs(*shape, dtype, seed=sum(shape)))


@pytest.mark.parametrize("H", [1, 24, 100])
def test_beam_state_widths(H):
    check_beam(*beam_inputs(3, 4, 300, "bf16", seed=1, H=H, L=3))
    check_beam(*beam_inputs(3, 4, 300, "f32", seed=1, H=H, L=1), alpha=0.0)


def test_beam_one_state_or_none():
    logits, scores, fin, lengths, h, c = beam_inputs(2, 3, 100, "f32", seed=2)
    check_beam(logits, scores, fin, lengths, h, None)
    check_beam(logits, scores, fin, lengths, None, c)
    check_beam(logits, scores, fin, lengths)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_beam_ties_go_to_the_lowest_index(dtype):
    logits, scores, fin, lengths, h, c = beam_inputs(2, 4, 3000, dtype, seed=3, finished=0)
    # equal beams, logits of few values: nearly everything is a tie, also between beams
    logits.copy_(logits[:, :1].expand_as(logits).clamp(min=-1, max=1).round())
    logits[..., 0] = -math.inf
    scores.fill_(-1.5)
    lengths.fill_(4)
    check_beam(logits, scores, fin, lengths, h, c)
    logits.fill_(0.25)
    check_beam(logits, scores, fin, lengths, h, c)


def test_beam_first_step_and_finished_sentences():
    logits, scores, fin, lengths, h, c = beam_inputs(4, 4, 500, "bf16", seed=4, finished=0)
    lengths.zero_()
    scores.zero_()
    scores[:, 1:] = -math.inf  # one beam lives
    fin[1] = 1                 # all finished, one of them live
    fin[2] = 1
    scores[2] = torch.tensor([-3.0, -1.0, -2.0, -1.0])  # all finished: reordered by score, ties by beam
    scores[3] = -math.inf      # none lives
    check_beam(logits, scores, fin, lengths, h, c)
    small = beam_inputs(2, 4, 4, "f32", seed=5, finished=0)
    small[0][..., 1:3] = -math.inf  # fewer live proposals than beams
    small[1][:, 1:] = -math.inf
    check_beam(*small)


def test_beam_rows_without_a_distribution():
    logits, scores, fin, lengths, h, c = beam_inputs(4, 3, 700, "f32", seed=6, finished=0)
    logits[0, 1, 77] = math.nan
    logits[1, 0, 5] = math.inf
    logits[2, 2] = -math.inf
    scores[3, 1] = math.nan
    s = decoder.prepare_beam(logits, scores, fin, lengths, eos=2, alpha=0.6)
    s.step()
    for b, k in ((0, 1), (1, 0), (2, 2), (3, 1)):
        assert k not in s.parents[b].tolist()
    clean = scores.clone()
    for b, k in ((0, 1), (1, 0), (2, 2), (3, 1)):
        clean[b, k] = -math.inf
    logits = torch.nan_to_num(logits, nan=0.0, posinf=0.0, neginf=-math.inf)
    want, _ = beam(logits, clean, fin, lengths, 2, 0.6)
    assert torch.equal(s.tokens.cpu(), want["tokens"]) and torch.equal(s.parents.cpu(), want["parents"])


def test_beam_strided_rows_and_extreme_logits():
    logits, scores, fin, lengths, h, c = beam_inputs(2, 5, 1003, "bf16", seed=7)
    wide = torch.full((2, 5, 1200), 50.0, dtype=torch.bfloat16, device=DEV)
    wide[..., 3:1006] = logits
    check_beam(wide[..., 3:1006], scores, fin, lengths, h, c)
    logits, scores, fin, lengths, h, c = beam_inputs(2, 3, 5000, "f32", seed=8)
    logits[0] *= 1e4
    logits[1] -= 3e38
    check_beam(logits, scores, fin, lengths, h, c, gap=0.0)


def test_beam_steps_capture():
    logits, scores, fin, lengths, h, c = beam_inputs(6, 4, 9001, "bf16", seed=9)
    s = decoder.prepare_beam(logits, scores, fin, lengths, eos=2, alpha=0.6, states=(h, c))
    s.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    outs = (s.tokens, s.parents, s.scores_out, s.finished_out, s.lengths_out, *s.states_out)
    for i in range(3):
        logits.copy_(logits.roll(17, -1))
        s.step()
        first = [x.clone() for x in outs]
        for x in outs:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, outs)), i


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["rising", "falling", "few", "late", "blocks"])
def test_beam_orders_of_logits(kind, dtype):
    """What the single pass over a row has to raise its bound for, or to give up on."""
    V = 40001
    logits, scores, fin, lengths, h, c = beam_inputs(1, 4, V, dtype, seed=10, finished=0)
    if kind in ("rising", "falling"):
        x = logits.sort(-1, descending=kind == "falling").values
    elif kind == "few":  # a vocabulary constrained to three tokens
        x = torch.full_like(logits, -math.inf)
        x[..., 5] = 1.0
        x[..., 7] = 0.5
        x[:, 1:, V - 1] = 2.0
    elif kind == "late":  # the best at the row's end, far above the rest
        x = logits.clone()
        x[..., -3:] = torch.tensor([90.0, 91.0, 89.0]).to(x)
    else:  # runs of equal values
        x = (torch.arange(V) // 1000 % 7).to(logits).expand_as(logits).clone()
    check_beam(x, scores, fin, lengths, h, c)


def test_beam_of_many_parts():
    check_beam(*beam_inputs(1, 16, 300001, "f32", seed=11, H=1024, L=2))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_beam_ties_far_apart_in_a_row(dtype):
    """A beam's best values are equal and lie in different parts of its row: lowest index first."""
    B, K, V = 40, 5, 32007
    logits, scores, fin, lengths, h, c = beam_inputs(B, K, V, dtype, seed=12, finished=0)
    g = torch.Generator().manual_seed(13)
    at = torch.randint(3, V, (B, K, 4), generator=g).to(DEV)
    logits.scatter_(2, at, 14.0)
    check_beam(logits, scores, fin, lengths, h, c)
