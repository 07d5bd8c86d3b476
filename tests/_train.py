"""64-bit definitions and rounding bounds for the training operators' tests. The bounds are elementwise:
u is half a step of the stored type relative to the value, A = 2^-24 per fp32 addition of a sum of
products (so n A times the sum of the products' magnitudes), F = 2^-20 for the fp32 exponential,
reciprocal and the few operations around them (under 16 roundings of 2^-24)."""
from __future__ import annotations

import torch

A, F = 2.0 ** -24, 2.0 ** -20
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def forward(x, gate, up, down, dtype):
    """(value, bound) of g, u and y for one group; all arguments float64."""
    un = half_step(dtype)
    n, i = x.shape[1], down.shape[0]
    g, u = x @ gate, x @ up
    ag, au = n * A * (x.abs() @ gate.abs()), n * A * (x.abs() @ up.abs())
    s = torch.sigmoid(g)
    h = g * s * u
    # |d SiLU| <= 1.1; both products' errors reach h, then h is rounded
    th = 1.1 * ag * (u.abs() + au) + (g * s).abs() * au + (un + F) * h.abs()
    y = h @ down
    ty = un * y.abs() + (1 + un) * (th @ down.abs() + i * A * (h.abs() @ down.abs()))
    return {"g": (g, un * g.abs() + (1 + un) * ag), "u": (u, un * u.abs() + (1 + un) * au), "y": (y, ty)}


def backward(x, gate, up, down, g, u, dy, dtype):
    un = half_step(dtype)
    n, i, rows = x.shape[1], down.shape[0], x.shape[0]
    s = torch.sigmoid(g)
    si = g * s
    dh = dy @ down.T
    adh = n * A * (dy.abs() @ down.abs().T)
    slope = s + si * (1 - s)
    du, dg, h = dh * si, dh * u * slope, si * u
    tdu = adh * si.abs() + (un + F) * du.abs()
    # the slope's two terms may cancel: its error is F times their magnitudes
    tdg = adh * (u * slope).abs() + un * dg.abs() + F * (dh * u).abs() * (s + si.abs())
    th = (un + F) * h.abs()

    def product(a, ta, b, extra=0.0):
        v = a @ b
        return v, un * v.abs() + (1 + un) * (ta @ b.abs() + extra * A * ((a.abs() + ta) @ b.abs()))
    dx = [product(dg, tdg, gate.T, 2 * i), product(du, tdu, up.T, 2 * i)]
    wt = {"dgate": product(dg.T, tdg.T, x, rows), "dup": product(du.T, tdu.T, x, rows)}
    out = {k: (v.T, t.T) for k, (v, t) in wt.items()}
    out["ddown"] = product(h.T, th.T, dy, rows)
    out["dx"] = (dx[0][0] + dx[1][0], dx[0][1] + dx[1][1])
    return out


def check(name, got, want, bound):
    """got within the bound of want everywhere (plus the type's smallest step, for values under its normal range)."""
    got = got.double()
    off = (got - want).abs()
    tiny = 2.0 ** -126
    worst = (off / (bound + tiny)).max().item() if off.numel() else 0.0
    assert torch.isfinite(got).all(), "%s: not finite" % name
    assert worst <= 1.0, "%s: %.3g of the bound" % (name, worst)
    return worst


def layout(counts, T, gen, device):
    """expert_offsets and slot_token for the given rows per expert, tokens drawn at random (repeats allowed)."""
    c = torch.tensor(counts)
    off = torch.zeros(len(counts) + 1, dtype=torch.int32)
    off[1:] = c.cumsum(0)
    slot = torch.randint(0, max(T, 1), (int(c.sum()),), generator=gen, dtype=torch.int32)
    return off.to(device), slot.to(device)


def chain_error(*lengths):
    """Relative Frobenius error of fp32 products of random signs chained one after the other (a product of the given
    reduction length each, whose operand is the one before), summed in rounds of 128 elements whose sums are added to
    a total. One addition rounds by 0.42 2^-24 of its result on average (uniform within half a step, the mantissa
    logarithmic), taken as 0.5; the partial sums of n terms have the mean square n / 2 of the whole's, so a round
    contributes 64 such squares, the total's K / 128 additions K / 256, and one more rounding forms an operand."""
    return 0.5 * A * sum(64 + n / 256 + 1 for n in lengths) ** 0.5
