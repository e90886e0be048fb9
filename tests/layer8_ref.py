"""64-bit references of the router and of int8 codes (test infrastructure)."""
import math

import torch

from layer_ref import EPS32

LOGIT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
NINF = -math.inf


def scores(l, score):
    """p of rows of 64-bit logits; a row with nothing on is 0."""
    if score == "sigmoid":
        return torch.special.expit(l)
    m = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(m > NINF, m, torch.zeros_like(m)))
    s = e.sum(1, keepdim=True)
    return torch.where(s > 0, e / s, torch.zeros_like(e))


def route(logits, top, bias=None, score="softmax", groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0):
    """(ids, weights, scores) token by token."""
    l = logits.double()
    tokens, experts = l.shape
    p = scores(l, score)
    b = torch.zeros(experts, dtype=torch.float64) if bias is None else bias.double()
    ids = torch.full((tokens, top), -1, dtype=torch.int32)
    w = torch.zeros((tokens, top), dtype=torch.float64)
    per = experts // groups
    for t in range(tokens):
        if torch.isnan(l[t]).any() or (score == "softmax" and (l[t] == math.inf).any()):
            w[t] = math.nan
            continue
        c = p[t] + b
        on = [e for e in range(experts) if l[t, e] > NINF and c[e] > NINF]
        if groups > 1:
            value = {}
            for g in range(groups):
                best = sorted((float(c[e]) for e in on if e // per == g), reverse=True)[:group_top]
                if best:
                    value[g] = sum(best)
            kept = sorted(value, key=lambda g: (-value[g], g))[:top_groups]
            on = [e for e in on if e // per in kept]
        # without a bias the order is the logits' own (p may round to equal numbers)
        order = sorted(on, key=lambda e: (-float(c[e] if bias is not None else l[t, e]), e))[:top]
        for j, e in enumerate(order):
            ids[t, j] = e
            w[t, j] = p[t, e]
    if renorm and score == "softmax":  # shares of the chosen alone: their scores may all round to 0
        v = torch.where(ids >= 0, l.gather(1, ids.long().clamp(min=0)), torch.full_like(w, NINF))
        w = torch.where(torch.isnan(w), w, torch.nan_to_num(scores(v, score)))
    elif renorm:
        s = w.sum(1, keepdim=True)
        w = torch.where(s > 0, w / s, torch.where(torch.isnan(s), w, torch.zeros_like(w)))
    return ids, w * scale, p


def score_error(logits, score):
    """Relative error of a token's scores in fp32: a softmax's exponential of a difference (rounded: |l - m| half
    steps) and its sum of up to 64 terms a lane and 6 steps over the lanes; a sigmoid's exponential and division."""
    l = logits.double()
    if score == "sigmoid":
        return torch.full((l.shape[0], 1), 12 * EPS32, dtype=torch.float64)
    far = l.clamp(min=-90.0)
    far = torch.where(torch.isfinite(far), far, torch.zeros_like(far))
    spread = far.amax(1, keepdim=True) - far.amin(1, keepdim=True)
    return (2 * spread + l.shape[1] / 64 + 24) * EPS32


def route_grad(dweights, logits, ids, score="softmax", renorm=True, scale=1.0):
    """(dlogits, the sum of its terms' magnitudes) by the formulas."""
    l = logits.double()
    p = scores(l, score)
    d, size = torch.zeros_like(l), torch.zeros_like(l)
    for t in range(l.shape[0]):
        on = [(j, int(e)) for j, e in enumerate(ids[t].tolist()) if 0 <= e < l.shape[1]]
        g = {j: scale * float(dweights[t, j]) for j, _ in on}
        total = sum(float(p[t, e]) for _, e in on)
        if renorm:
            a = {j: (float(p[t, e]) / total if total > 0 else 0.0) for j, e in on}
            mean = sum(a[j] * g[j] for j, _ in on)
            mean_size = sum(a[j] * abs(g[j]) for j, _ in on)
            for j, e in on:
                slope = 1.0 if score == "softmax" else 1.0 - float(p[t, e])
                d[t, e] += a[j] * slope * (g[j] - mean)
                size[t, e] += a[j] * slope * (abs(g[j]) + mean_size)
        elif score == "softmax":
            mean = sum(float(p[t, e]) * g[j] for j, e in on)
            mean_size = sum(float(p[t, e]) * abs(g[j]) for j, e in on)
            for j, e in on:
                d[t, e] += p[t, e] * g[j]
                size[t, e] += p[t, e] * abs(g[j])
            d[t] -= p[t] * mean
            size[t] += p[t] * mean_size
        else:
            for j, e in on:
                d[t, e] += p[t, e] * (1 - p[t, e]) * g[j]
                size[t, e] += p[t, e] * (1 - p[t, e]) * abs(g[j])
    return d, size


def codes(x, group):
    """(codes, scale) of rows by the definition in fp32 (IEEE division, ties to even)."""
    cols = x.shape[1]
    width = group or cols
    c = torch.zeros(x.shape, dtype=torch.int8)
    s = torch.zeros((x.shape[0], -(-cols // width)), dtype=torch.float32)
    for i in range(s.shape[1]):
        b = x[:, i * width:(i + 1) * width].float()
        # (amax drops no NaN)
        scale = b.abs().amax(1) / torch.tensor(127.0)
        s[:, i] = scale
        usable = (scale > 0) & torch.isfinite(scale)
        q = torch.round(b / torch.where(usable, scale, torch.ones_like(scale))[:, None]).clamp(-127, 127)
        c[:, i * width:(i + 1) * width] = torch.where(usable[:, None], q, torch.zeros_like(q)).to(torch.int8)
    return c, s


def values(c, s, group):
    """What codes stand for, in 64 bits."""
    width = group or c.shape[1]
    return c.double() * s.double().repeat_interleave(width, dim=1)[:, :c.shape[1]]
