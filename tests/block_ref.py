"""The operators around the dispatch in 64 bits, on CPU tensors: from their formulas, one line for each."""
import math

import numpy as np
import torch

F64 = torch.float64


def half_step(dtype) -> float:
    """The most a rounding to dtype is off, relative to the value."""
    return torch.finfo(dtype).eps / 2


def norm(x, residual, weight, eps):
    """h in the inputs' dtype (the sum of two values of it, rounded once) and y in 64 bits."""
    h = x if residual is None else (x.to(F64) + residual.to(F64)).to(x.dtype)
    f = h.to(F64)
    return h, f / (f.square().mean(1, keepdim=True) + eps).sqrt() * weight.to(F64)


def norm_grad(dy, dy2, h, weight, eps, dres):
    """dx, dw, and what bounds their rounding errors: the sums of the terms' sizes."""
    d, f, w = dy.to(F64), h.to(F64), weight.to(F64)
    if dy2 is not None:
        d = d + dy2.to(F64)
    n = f.shape[1]
    s = 1 / (f.square().sum(1, keepdim=True) / n + eps).sqrt()
    dot, size = (d * w * f).sum(1, keepdim=True) / n, (d * w * f).abs().sum(1, keepdim=True) / n
    dx = s * (d * w - f * s * s * dot)
    terms = s * ((d * w).abs() + f.abs() * s * s * size)
    if dres is not None:
        dx, terms = dx + dres.to(F64), terms + dres.to(F64).abs()
    return dx, terms, (d * f * s).sum(0), (d * f * s).abs().sum(0)


def scores(z, score):
    """64-bit scores; 0 for a masked expert (-inf or NaN), shares of a +inf one that is the softmax's limit."""
    z = torch.where(z.isnan(), torch.full_like(z, -math.inf), z.to(F64))
    masked = z == -math.inf
    if score == "sigmoid":
        return torch.where(masked, torch.zeros_like(z), 1 / (1 + torch.exp(-z)))
    top = z.max(1, keepdim=True).values
    e = torch.where(z == top, torch.ones_like(z), torch.exp(z - top))
    e = torch.where(masked, torch.zeros_like(z), e)
    return e / e.sum(1, keepdim=True).clamp(min=1e-300)


def route(logits, topk, score, bias=None, groups=1, top_groups=1, renormalise=False, scale=1.0):
    """ids and gates, one token after the other."""
    z = logits.to(F64)
    s = scores(z, score)
    scored = bias is not None or top_groups < groups
    key = s + (bias.to(F64) if bias is not None else 0) if scored else z
    key = torch.where(z.isnan() | (z == -math.inf) | key.isnan(), torch.full_like(key, -math.inf), key)
    tokens, experts = z.shape
    per = experts // groups
    ids = np.full((tokens, topk), -1, dtype=np.int32)
    for t in range(tokens):
        k = key[t].tolist()
        if top_groups < groups:
            strength = []
            for g in range(groups):
                best = sorted((v for v in k[g * per:(g + 1) * per] if v > -math.inf), reverse=True)[:2]
                strength.append(sum(best) if best else -math.inf)
            kept = sorted(range(groups), key=lambda g: (-strength[g], g))[:top_groups]
            k = [v if e // per in kept else -math.inf for e, v in enumerate(k)]
        order = sorted((e for e in range(experts) if k[e] > -math.inf), key=lambda e: (-k[e], e))[:topk]
        ids[t, :len(order)] = order
    ids = torch.from_numpy(ids)
    return ids, gates(z, ids, score, renormalise, scale)


def gates(z, ids, score, renormalise, scale):
    """The gates of given ids, in 64 bits; differentiable for z.  Renormalised sigmoids by their logarithms, so that they
    hold where every one of them underflows."""
    at = ids.long().clamp(min=0)
    there = ids >= 0
    if renormalise:
        chosen = z.gather(1, at)
        lg = chosen if score == "softmax" else torch.nn.functional.logsigmoid(chosen)
        lg = torch.where(there, lg, torch.full_like(lg, -math.inf))
        inf = (lg == math.inf).any(1, keepdim=True)
        lg = torch.where(inf, torch.where(lg == math.inf, torch.zeros_like(lg), torch.full_like(lg, -math.inf)), lg)
        lg = torch.where(there.any(1, keepdim=True), lg, torch.zeros_like(lg))
        g = torch.softmax(lg, 1)
    elif z.requires_grad:
        g = (torch.softmax(z, 1) if score == "softmax" else torch.sigmoid(z)).gather(1, at)
    else:
        g = scores(z, score).gather(1, at)
    return torch.where(there, g * scale, torch.zeros_like(g))


def philox_bits(n, seed, first=0):
    """16 random bits of each of n elements from element `first` on (a multiple of 8), in numpy's uint64."""
    mask = np.uint64(0xFFFFFFFF)
    w = lambda v, i: np.uint64((int(v) >> (32 * i)) & 0xFFFFFFFF)  # noqa: E731
    g = np.arange((n + 7) // 8, dtype=np.uint64) + np.uint64(first // 8)
    c = [g & mask, g >> np.uint64(32), np.full_like(g, w(seed[1], 0)), np.full_like(g, w(seed[1], 1))]
    k = [w(seed[0], 0), w(seed[0], 1)]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ k[0], b & mask, (a >> np.uint64(32)) ^ c[3] ^ k[1], a & mask]
        k = [(k[0] + np.uint64(0x9E3779B9)) & mask, (k[1] + np.uint64(0xBB67AE85)) & mask]
    out = np.empty((len(g), 8), dtype=np.int64)
    for i, v in enumerate(c):
        out[:, 2 * i] = (v & np.uint64(0xFFFF)).astype(np.int64)
        out[:, 2 * i + 1] = (v >> np.uint64(16)).astype(np.int64)
    return torch.from_numpy(out.reshape(-1)[:n])
