"""64-bit definitions of the gate, the Newton-Schulz steps and the Muon step, and how far their kernels may be off."""
from __future__ import annotations

import math

import numpy as np
import torch

F = 2.0 ** -20  # an fp32 exponential, reciprocal and the few operations around them: under 16 roundings of 2^-24
NS = (3.4445, -4.7750, 2.0315)


def gate_row(logits, bias, k, score, groups, top_groups, group_top, renormalize, scale):
    """(experts, weights) of one token by the definition, in 64 bits; finite or -inf logits."""
    l = np.asarray(logits, dtype=np.float64)
    E = len(l)
    with np.errstate(over="ignore"):
        if score == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-l))
        else:
            top = l.max()
            s = np.exp(l - top) / np.exp(l - top).sum() if top > -np.inf else np.zeros(E)
    on = [e for e in range(E) if l[e] > -np.inf and (bias is None or bias[e] > -np.inf)]
    c = {e: s[e] + (0.0 if bias is None else float(bias[e])) for e in on}
    if groups > 1:
        size = E // groups
        worth = []
        for g in range(groups):
            best = sorted((c[e] for e in on if e // size == g), reverse=True)[:group_top]
            worth.append((-sum(best) if best else np.inf, g))
        kept = {g for _, g in sorted(worth)[:top_groups]}
        on = [e for e in on if e // size in kept]
    order = c if bias is not None else l  # the order of the scores, also where they are 0 in 64 bits
    chosen = sorted(sorted(on, key=lambda e: (-order[e], e))[:k])
    w = np.array([s[e] for e in chosen])
    if renormalize and len(chosen):
        w = w / w.sum()
    return chosen + [-1] * (k - len(chosen)), list(scale * w) + [0.0] * (k - len(chosen))


def gate_gradient(logits, idx, dw, score, renormalize, scale):
    """(dlogits, bound) in 64 bits; the bound is F times the magnitudes that are added."""
    l = logits.double()
    on = l > -math.inf
    T, E = l.shape
    e = idx.long()
    here = (e >= 0) & (e < E)
    e = e.clamp(0, E - 1)
    here &= on.gather(1, e)
    if score == "sigmoid":
        s, rest = torch.sigmoid(l), torch.sigmoid(-l)
    else:
        s, rest = torch.softmax(l.masked_fill(~on, -1e30), 1).masked_fill(~on, 0.0), torch.ones_like(l)
    d = torch.where(here, dw.double(), 0.0)
    c = torch.where(here, s.gather(1, e), 0.0)
    if score == "softmax" and not renormalize:
        spread = torch.zeros_like(l).scatter_add_(1, e, d)
        size = torch.zeros_like(l).scatter_add_(1, e, d.abs())
        mean, most = (c * d).sum(1, keepdim=True), (c * d.abs()).sum(1, keepdim=True)
        return scale * s * (spread - mean), F * abs(scale) * s * (size + most)
    if renormalize:
        r = c / c.sum(1, keepdim=True).clamp(min=1e-300)
        mean, most = (r * d).sum(1, keepdim=True), (r * d.abs()).sum(1, keepdim=True)
    else:
        r, mean, most = c, 0.0, 0.0
    f = scale * r * rest.gather(1, e) * here
    out = torch.zeros_like(l).scatter_add_(1, e, f * (d - mean))
    return out, F * torch.zeros_like(l).scatter_add_(1, e, f.abs() * (d.abs() + most))


def newton_schulz(g, steps=5, coef=NS, eps=1e-7):
    """A stack [count, rows, cols] in 64 bits."""
    a, b, c = coef
    x = g.double()
    norm = x.square().sum((1, 2), keepdim=True).sqrt() + eps
    x = torch.where(norm > 0, x / norm, 0.0)
    wide = x.shape[1] <= x.shape[2]
    if not wide:
        x = x.transpose(1, 2).contiguous()
    for _ in range(steps):
        A = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * A + c * torch.bmm(A, A), x)
    return x if wide else x.transpose(1, 2).contiguous()


def rounded_steps(g, steps=5, coef=NS, eps=1e-7):
    """The same with the roundings that the 16-bit products' operands take and nothing else: x to fp16 in the products,
    to a pair of them beside; A and C to fp16 but for their diagonals; in the last step x to fp16 alone, and C's diagonal.
    In 64 bits otherwise."""
    a, b, c = coef
    S = 4096.0
    x = g.double()
    norm = x.square().sum((1, 2), keepdim=True).sqrt() + eps
    x = torch.where(norm > 0, x * (S / norm), 0.0)
    wide = x.shape[1] <= x.shape[2]
    if not wide:
        x = x.transpose(1, 2).contiguous()
    half = lambda t: t.half().double()  # noqa: E731
    diagonal = lambda t: torch.diagonal(t, dim1=1, dim2=2).clone()  # noqa: E731
    bare = lambda t: half(t - torch.diag_embed(diagonal(t)))  # noqa: E731
    for i in range(steps):
        h = half(x)
        x = h + half(x - h) if i + 1 < steps else h
        A = torch.bmm(h, h.transpose(1, 2).contiguous()) / S
        d, A = diagonal(A) / S, bare(A)
        A2 = torch.bmm(A, A) / S
        C = b * A + c * ((d[:, :, None] + d[:, None, :]) * A + A2)
        dc, C = b * d + c * (d * d + diagonal(A2) / S), bare(C)
        dc = a + dc if i + 1 < steps else half((a + dc) * S) / S
        x = dc[:, :, None] * x + torch.bmm(C, h) / S
    x = x / S
    return x if wide else x.transpose(1, 2).contiguous()


def plain_steps(g, steps=5, coef=NS, eps=1e-7):
    """The same in fp32."""
    a, b, c = coef
    x = g.float()
    norm = x.double().square().sum((1, 2), keepdim=True).sqrt() + eps
    x = torch.where(norm > 0, x / norm, 0.0).float()
    wide = x.shape[1] <= x.shape[2]
    if not wide:
        x = x.transpose(1, 2).contiguous()
    for _ in range(steps):
        A = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * A + c * torch.bmm(A, A), x)
    return (x if wide else x.transpose(1, 2).contiguous()).double()


def off(x, y):
    """Each matrix's error relative to its norm."""
    n = y.square().sum((1, 2)).sqrt()
    d = (x.double() - y).square().sum((1, 2)).sqrt()
    return torch.where(n > 0, d / n, d)


def step_errors(g, dtype, **kw):
    """(O in 64 bits, the error that each of its matrices may have before it is rounded to its own type).
    bf16: twice that of rounded_steps: the kernel adds fp32 sums, 13 bits below the operands' rounding, which move
    single operands to the other neighbour. fp32: the operands of 22 bits where plain_steps has 24, and the product of
    the two low parts left out: 4 times that of plain_steps, and as much again for what differs by chance; at
    least 2^-20, 16 roundings of 2^-24 for the few sums of small matrices."""
    want = newton_schulz(g, **kw)
    if dtype == torch.bfloat16:
        return want, 2 * off(rounded_steps(g, **kw), want)
    return want, (8 * off(plain_steps(g, **kw), want)).clamp(min=2.0 ** -20)
