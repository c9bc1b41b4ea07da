"""The decoder operators' workloads: what runs, on which inputs, and what it costs at least.

Three operators of an encoder-decoder recurrent network, in four uses:

  fwd     attention of a decoder's outputs over an encoder's outputs (teacher-forced decoding, scoring)
  train   the same with its gradients: one forward and one backward
  decode  attention of the tokens of one step (one token, or the beams of a sentence, which share its encoder outputs)
  beam    one step of beam search: selection over beams and vocabulary, and the reordering of the recurrent states

``run`` computes them in plain torch operations where ``own`` is false, and through the library where it is true.
"""
import math

import torch

own = False

DEVICE = "cuda:0"
EOS = 2
ALPHA = 0.6  # exponent of the length penalty
SPREAD = {"none": 1.0, "lengths": 0.75, "holes": 0.8}  # mean share of the keys that the mask leaves


def _attn(use, name, B, Tq, S, Hq, Hkv, D, dtype, layout, mask):
    return {"name": name, "use": use, "B": B, "Tq": Tq, "S": S, "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": dtype,
            "layout": layout, "mask": mask}


def _beam(name, B, K, V, dtype, L, H):
    return {"name": name, "use": "beam", "B": B, "K": K, "V": V, "dtype": dtype, "L": L, "H": H}


def listed():
    return [
        # the smallest: two heads over the outputs of a 128-wide fp32 layer of 16 steps; latency counts
        _attn("fwd", "fwd f32 2x64 T16", 8, 16, 16, 2, 2, 64, "f32", "tbh", "none"),
        # scoring a batch of ragged sentences with a 256-wide bf16 stack, sources longer than targets
        _attn("fwd", "fwd bf16 4x64 ragged", 64, 200, 331, 4, 4, 64, "bf16", "tbh", "lengths"),
        # long documents through a 4096-wide stack: the largest product
        _attn("fwd", "fwd bf16 32x128 long", 8, 2048, 4096, 32, 32, 128, "bf16", "bth", "none"),
        # a training step of the 512-wide fp32 stack on ragged sentences
        _attn("train", "train f32 8x64 ragged", 64, 100, 120, 8, 8, 64, "f32", "tbh", "lengths"),
        # shared key heads, a head size that is no power of two, single source positions left out
        _attn("train", "train bf16 16/4x80 holes", 32, 50, 777, 16, 4, 80, "bf16", "tbh", "holes"),
        # a training step on long sequences of a 1536-wide bf16 layer
        _attn("train", "train bf16 12x128 long", 4, 2048, 3001, 12, 12, 128, "bf16", "tbh", "lengths"),
        # greedy decoding of one sentence: one token
        _attn("decode", "decode bf16 1 token", 1, 1, 100, 8, 8, 64, "bf16", "bth", "none"),
        # beam search over a batch of sentences: five beams read one sentence's encoder outputs
        _attn("decode", "decode bf16 5 beams", 32, 5, 1000, 8, 8, 64, "bf16", "tbh", "lengths"),
        # beams over whole books: memory traffic is all
        _attn("decode", "decode bf16 8 beams long", 16, 8, 32768, 32, 8, 128, "bf16", "bth", "none"),
        # one sentence, a small vocabulary
        _beam("beam f32 1x4x8000", 1, 4, 8000, "f32", 1, 128),
        # a translation batch: an odd vocabulary, four layers of 512
        _beam("beam bf16 64x5x32007", 64, 5, 32007, "bf16", 4, 512),
        # a large batch over a large vocabulary, states of a 1536-wide stack
        _beam("beam bf16 256x8x131072", 256, 8, 131072, "bf16", 4, 1536),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {c["name"]: work(c) for c in listed()}
    while True:
        use = rng.choice(("fwd", "train", "decode", "beam"))
        dtype = rng.choice(("bf16", "bf16", "f32"))
        if use == "beam":
            c = _beam("", _log(rng, 1, 256), rng.choice((1, 2, 3, 4, 5, 8, 10, 16)), _log(rng, 1000, 150000), dtype,
                      rng.choice((1, 2, 4)), 8 * _log(rng, 16, 256))
            top = most["beam bf16 256x8x131072"]
        else:
            hkv = rng.choice((1, 2, 4, 8, 12, 16))
            g = rng.choice((1, 1, 1, 2, 4, 8))
            d = rng.choice((32, 64, 64, 64, 80, 96, 128, 128, 200, 256))
            layout = rng.choice(("tbh", "bth"))
            mask = rng.choice(("none", "lengths", "lengths", "holes"))
            if use == "decode":
                c = _attn(use, "", _log(rng, 1, 128), rng.choice((1, 1, 2, 4, 5, 8)), _log(rng, 20, 65536), hkv * g,
                          hkv, d, dtype, layout, mask)
                top = most["decode bf16 8 beams long"]
            else:
                c = _attn(use, "", _log(rng, 2, 64), _log(rng, 10, 2500), _log(rng, 10, 4500), hkv * g, hkv, d, dtype,
                          layout, mask)
                top = most["fwd bf16 32x128 long" if use == "fwd" else "train bf16 12x128 long"]
        del c["name"]
        w = work(c)
        # fp32 products cost this card about 16 times as much as bf16 ones
        dear = 16 if c["dtype"] == "f32" and use in ("fwd", "train") else 1
        if w["flops"] * dear <= top["flops"] and w["bytes"] <= max(top["bytes"], top["flops"] / 500):
            return c


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["use"] == "beam":
        rows = case["B"] * case["K"]
        live = 0.85  # finished beams need no logits
        states = 2 * case["L"] * rows * case["H"] * (size + 4)
        return {"bytes": rows * case["V"] * size * live + states + rows * 34, "flops": 4 * rows * case["V"] * live}
    B, Tq, Hq, Hkv, D = (case[k] for k in ("B", "Tq", "Hq", "Hkv", "D"))
    S = case["S"] * (1.0 if case["mask"] == "holes" else SPREAD[case["mask"]])
    q, kv, pairs = B * Tq * Hq * D, B * S * Hkv * D, B * Tq * Hq * case["S"] * SPREAD[case["mask"]]
    mask = B * case["S"] if case["mask"] == "holes" else 4 * B if case["mask"] == "lengths" else 0
    if case["use"] == "train":
        return {"bytes": (4 * q + 4 * kv) * size + mask, "flops": 14 * pairs * D}
    return {"bytes": (2 * q + 2 * kv) * size + 4 * B * Tq * Hq + mask, "flops": 4 * pairs * D}


# ---------------------------------------------------------------------------------------------------------------------
# inputs


def _inputs(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

    def normal(*shape, by=1.0):
        return torch.randn(shape, generator=g, device=DEVICE).mul_(by).to(dt)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEVICE)

    B = case["B"]
    if case["use"] == "beam":
        K, V, L, H = case["K"], case["V"], case["L"], case["H"]
        logits = normal(B, K, V, by=2.5)
        logits[..., 0] = -math.inf  # padding is never produced
        lengths = 10 + (20 * uniform(B, K)).int()
        scores = -lengths * (0.2 + uniform(B, K))
        return {"logits": logits, "scores": scores, "finished": (uniform(B, K) < 0.15).to(torch.uint8),
                "lengths": lengths, "h": normal(L, B * K, H, by=0.5),
                "c": torch.randn((L, B * K, H), generator=g, device=DEVICE)}

    def tensor(T, heads, by=1.0):
        if case["layout"] == "tbh":  # as the recurrence writes its outputs: step, sentence, feature
            return normal(T, B, heads, case["D"], by=by).transpose(0, 1)
        return normal(B, T, heads, case["D"], by=by)

    Tq, S = case["Tq"], case["S"]
    s = {"q": tensor(Tq, case["Hq"], 1.5), "k": tensor(S, case["Hkv"]), "v": tensor(S, case["Hkv"]), "kv_len": None,
         "key_mask": None}
    if case["mask"] == "lengths":
        n = (S * (0.5 + 0.5 * uniform(B))).int().clamp(1, S)
        if B >= 8:
            n[B // 3] = 0  # a sentence with no source left
        s["kv_len"] = n
    elif case["mask"] == "holes":
        s["key_mask"] = (uniform(B, S) < 0.8).to(torch.uint8)
    if case["use"] == "train":
        s["do"] = tensor(Tq, case["Hq"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["use"] = case["use"]
    if own:
        from stacked_lstm_forward_amd import decoder

        if case["use"] == "beam":
            s["problem"] = decoder.prepare_beam(s["logits"], s["scores"], s["finished"], s["lengths"], eos=EOS,
                                                alpha=ALPHA, states=(s["h"], s["c"]))
        else:
            s["problem"] = decoder.prepare_attn(s["q"], s["k"], s["v"], kv_len=s["kv_len"], key_mask=s["key_mask"],
                                                train=case["use"] == "train")
    return s


# ---------------------------------------------------------------------------------------------------------------------
# the pass


def run(s):
    if own:
        p = s["problem"]
        if s["use"] == "beam":
            p.step()
            return {"tokens": p.tokens, "parents": p.parents, "scores": p.scores_out, "finished": p.finished_out,
                    "lengths": p.lengths_out, "h": p.states_out[0], "c": p.states_out[1]}
        p.forward()
        if s["use"] != "train":
            return {"o": p.o, "lse": p.lse}
        p.backward(s["do"])
        return {"o": p.o, "lse": p.lse, "dq": p.dq, "dk": p.dk, "dv": p.dv}
    if s["use"] == "beam":
        return _plain_beam(s)
    return _plain_attention(s)


def _plain_attention(s):
    q, k, v = s["q"], s["k"], s["v"]
    (B, Tq, Hq, D), (S, Hkv) = q.shape, k.shape[1:3]
    scale = 1.0 / math.sqrt(D)

    def rows(x):  # [B, T, H, D] -> [B * Hkv, G * T, D], fp32
        return x.float().transpose(1, 2).reshape(B * Hkv, -1, D)

    def back(x, T):  # and back, in the input's type
        return x.view(B, -1, T, D).transpose(1, 2).to(q.dtype)

    qf, kf, vf = rows(q), rows(k), rows(v)
    keep = None
    if s["kv_len"] is not None:
        keep = torch.arange(S, device=q.device) < s["kv_len"][:, None]
    elif s["key_mask"] is not None:
        keep = s["key_mask"] != 0
    p = torch.bmm(qf, kf.transpose(1, 2)).mul_(scale)
    if keep is not None:
        p.view(B, -1, S).masked_fill_(~keep[:, None], -math.inf)
    m = p.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(l == 0, 1.0, l))
    o = torch.bmm(p, vf)
    lse = (m + l.log()).view(B, Hq, Tq)
    out = {"o": back(o, Tq), "lse": lse}
    if "do" in s:
        do = rows(s["do"])
        out["dv"] = back(torch.bmm(p.transpose(1, 2), do), S)
        ds = torch.bmm(do, vf.transpose(1, 2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
        out["dq"] = back(torch.bmm(ds, kf), Tq)
        out["dk"] = back(torch.bmm(ds.transpose(1, 2), qf), S)
    return out


def _plain_beam(s):
    logits, scores, finished, lengths = s["logits"], s["scores"], s["finished"] != 0, s["lengths"]
    B, K, V = logits.shape
    # 64 bits: candidates of different beams may lie closer together than fp32 tells apart
    x = logits.double()
    m = x.amax(-1, keepdim=True)
    lse = m + (x - m).exp_().sum(-1, keepdim=True).log()
    cand = x.sub_(lse).add_(scores.double()[..., None])
    cand.masked_fill_(finished[..., None], -math.inf)
    cand[..., EOS] = torch.where(finished, scores.double(), cand[..., EOS])
    longer = lengths + (~finished).int()
    rank = (cand / ((5.0 + longer.double()) / 6.0).pow(ALPHA)[..., None]).view(B, K * V)
    # the K best; among equals the lowest index
    least = rank.topk(K, -1).values[:, -1:]
    over, level = rank > least, rank == least
    level &= level.cumsum(-1, dtype=torch.int32) <= K - over.sum(-1, keepdim=True)
    index = torch.arange(K * V, 0, -1, device=rank.device, dtype=torch.int32)
    at = K * V - torch.where(over | level, index, 0).topk(K, -1).values.long()
    order = rank.gather(-1, at).sort(dim=-1, descending=True, stable=True).indices
    at = at.gather(-1, order)
    parents, tokens = at // V, at % V
    done = finished.gather(-1, parents) | (tokens == EOS)
    row = (parents + K * torch.arange(B, device=at.device)[:, None]).view(-1)
    return {"tokens": tokens.int(), "parents": parents.int(), "scores": cand.view(B, K * V).gather(-1, at).float(),
            "finished": done.to(torch.uint8), "lengths": longer.gather(-1, parents), "h": s["h"][:, row],
            "c": s["c"][:, row]}


# ---------------------------------------------------------------------------------------------------------------------
# the definition, in 64 bits


def exact(case, seed):
    s = _inputs(case, seed)
    if case["use"] == "beam":
        return _exact_beam(case, s)
    B, Hq, D = case["B"], case["Hq"], case["D"]
    G = Hq // case["Hkv"]
    o = torch.zeros((B, case["Tq"], Hq, D), dtype=torch.float64, device=DEVICE)
    lse = torch.full((B, Hq, case["Tq"]), -math.inf, dtype=torch.float64, device=DEVICE)
    grads = {n: torch.zeros(s[n].shape, dtype=torch.float64, device=DEVICE) for n in "qkv"}
    for b in range(B):
        at = torch.arange(case["S"], device=DEVICE)
        if s["kv_len"] is not None:
            at = at[: int(s["kv_len"][b])]
        if s["key_mask"] is not None:
            at = at[s["key_mask"][b].bool()]
        if len(at) == 0:
            continue
        for j in range(case["Hkv"]):
            heads = slice(j * G, j * G + G)
            q = s["q"][b, :, heads].double().reshape(-1, D)  # rows: step, then head of the group
            k, v = s["k"][b, at, j].double(), s["v"][b, at, j].double()
            z = q @ k.t().contiguous() / math.sqrt(D)
            n = torch.logsumexp(z, -1, keepdim=True)
            p = torch.exp(z - n)
            o[b, :, heads] = (p @ v).view(-1, G, D)
            lse[b, heads] = n.view(-1, G).t()
            if case["use"] == "train":
                do = s["do"][b, :, heads].double().reshape(-1, D)
                dp = do @ v.t().contiguous()
                dz = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(D)
                grads["q"][b, :, heads] = (dz @ k).view(-1, G, D)
                grads["k"][b, at, j] = dz.t().contiguous() @ q
                grads["v"][b, at, j] = p.t().contiguous() @ do
    out = {"o": o, "lse": lse}
    if case["use"] == "train":
        out.update({"d" + n: x for n, x in grads.items()})
    return out


def _exact_beam(case, s):
    B, K, V = case["B"], case["K"], case["V"]
    scores = torch.empty((B, K), dtype=torch.float64, device=DEVICE)
    row = torch.empty((B, K), dtype=torch.int64, device=DEVICE)
    for b in range(B):
        finished = s["finished"][b].bool()
        cand = torch.log_softmax(s["logits"][b].double(), -1) + s["scores"][b].double()[:, None]
        cand[finished] = -math.inf
        cand[finished, EOS] = s["scores"][b].double()[finished]
        n = s["lengths"][b].double() + (~finished).double()
        rank = (cand / torch.exp(ALPHA * torch.log((5 + n) / 6))[:, None]).reshape(-1)
        best = torch.sort(rank, descending=True, stable=True).indices[:K]
        scores[b] = cand.reshape(-1)[best]
        row[b] = b * K + best // V
    row = row.view(-1)
    return {"tokens": None, "parents": None, "scores": scores, "finished": None, "lengths": None,
            "h": s["h"][:, row].double(), "c": s["c"][:, row].double()}
