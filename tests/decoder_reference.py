"""Plain 64-bit forms of the decoder operators, and how far the kernels' results may be from them.

A rounding to a type is off by at most u = eps / 2 of the value.  The kernels round p and dz to the
tensors' type for their products, o, dq, dk, dv on output, and use the rounded o in delta; sums and
statistics are fp32.  `attention` returns each result with the bound that follows, element by element.
"""
import math

import torch


def keys(B, S, kv_len, key_mask):
    keep = torch.ones(B, S, dtype=torch.bool)
    if kv_len is not None:
        keep &= torch.arange(S)[None] < kv_len.cpu()[:, None]
    if key_mask is not None:
        keep &= key_mask.cpu().bool()
    return keep


def attention(q, k, v, kv_len=None, key_mask=None, dout=None, scale=None):
    """{name: (value, bound)} in float64 on the CPU; layouts as the library's."""
    u = torch.finfo(q.dtype).eps / 2
    w = 2.0 ** -24
    B, Tq, Hq, D = q.shape
    S, Hkv = k.shape[1:3]
    G = Hq // Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    keep = keys(B, S, kv_len, key_mask)
    qd = q.cpu().double().transpose(1, 2)  # [B, Hq, Tq, D]

    def wide(x):  # [B, S, Hkv, D] -> [B, Hq, S, D], other positions than the keys' never used
        x = torch.where(keep[:, :, None, None], x.cpu().double(), 0.0)
        return x.transpose(1, 2).repeat_interleave(G, 1).contiguous()

    def narrow(x):  # sums over the heads that share a key head
        return x.view(B, Hkv, G, S, D).sum(2).transpose(1, 2)

    def t(x):
        return x.transpose(-1, -2).contiguous()

    kd, vd = wide(k), wide(v)
    z = torch.where(keep[:, None, None], scale * (qd @ t(kd)), -math.inf)
    lse = torch.logsumexp(z, -1) if S else torch.full((B, Hq, Tq), -math.inf, dtype=torch.float64)
    p = torch.exp(z - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    o = p @ vd
    # fp32: the scores' sums of D products, their scaling and the exponential's argument; sums over S
    dz_abs = w * ((D + 4) * scale * (qd.abs() @ t(kd.abs())).amax(-1, keepdim=True) if S else torch.zeros(1))
    rel = dz_abs + w * (2 * lse.abs().clamp(max=1e30)[..., None] + S + 16) if S else torch.zeros(1, dtype=torch.float64)
    rel = torch.nan_to_num(rel, posinf=0.0)
    up = u if q.dtype != torch.float32 else 0.0  # p and dz are rounded in 16-bit products only
    spread = p @ vd.abs()
    e_o = (up + rel) * spread + u * o.abs()
    out = {"o": (o.transpose(1, 2), e_o.transpose(1, 2)),
           "lse": (lse, (rel.expand(*lse.shape, 1)[..., 0] if S else torch.zeros_like(lse)) + w * lse.abs().clamp(max=1e30))}
    if dout is not None:
        dd = dout.cpu().double().transpose(1, 2)
        delta = (dd * o).sum(-1, keepdim=True)
        e_delta = (dd.abs() * (e_o + w * (D + 2) * o.abs())).sum(-1, keepdim=True)
        dp = dd @ t(vd)
        e_dp = w * (D + 2) * (dd.abs() @ t(vd.abs()))
        dz = p * (dp - delta)
        e_dz = p * (e_dp + e_delta) + (up + 2 * rel) * dz.abs()
        n = w * (G * Tq + S + 8)  # the fp32 sums over rows or keys
        dq, dk, dv = scale * (dz @ kd), scale * (t(dz) @ qd), t(p) @ dd
        b_dq = scale * ((e_dz + n * dz.abs()) @ kd.abs()) + u * dq.abs()
        b_dk = scale * (t(e_dz + n * dz.abs()) @ qd.abs())
        b_dv = t((up + rel + n) * p) @ dd.abs()
        dk, dv = narrow(dk), narrow(dv)
        out["dq"] = (dq.transpose(1, 2), b_dq.transpose(1, 2))
        out["dk"] = (dk, narrow(b_dk) + u * dk.abs())
        out["dv"] = (dv, narrow(b_dv) + u * dv.abs())
    return out


def beam(logits, scores, finished, lengths, eos, alpha):
    """tokens, parents, scores, finished, lengths [B, K] and the smallest gap between different ranks
    among each sentence's first K + 1 (float64, CPU)."""
    B, K, V = logits.shape
    fin = finished.cpu().bool()
    sc = scores.cpu().double()
    x = logits.cpu().double()
    cand = sc[..., None] + (x - torch.logsumexp(x, -1, keepdim=True))
    cand[fin] = -math.inf
    cand[..., eos] = torch.where(fin, sc, cand[..., eos])
    cand = torch.where(torch.isnan(cand) | torch.isinf(sc)[..., None], -math.inf, cand)
    n = lengths.cpu() + (~fin).int()
    rank = (cand / ((5 + n.double()) / 6).pow(alpha)[..., None]).view(B, K * V)
    top = torch.sort(rank, dim=-1, descending=True, stable=True)
    at = top.indices[:, :K]
    first = top.values[:, :K + 1]
    d = first[:, :-1] - first[:, 1:]
    d = d[torch.isfinite(d) & (d > 0)]
    parents, tokens = at // V, at % V
    return {"tokens": tokens.int(), "parents": parents.int(), "scores": cand.view(B, K * V).gather(1, at),
            "finished": (fin.gather(1, parents) | (tokens == eos)).to(torch.uint8),
            "lengths": n.gather(1, parents).int()}, float(d.min()) if d.numel() else math.inf
