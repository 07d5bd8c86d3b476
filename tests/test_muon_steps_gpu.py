"""Orthogonalisation and Muon steps with step counts and polynomials other than the usual ones, for every kind of kernel, on the GPU."""
import math

import pytest
import torch

from expert_ffn_layer_amd import native as N

from _gpu import say
from _muon import NS, newton_schulz, off, step_errors
from test_muon_gpu import DEV, DT, Step, gen_of, matrices, orthogonalize, verify, workspace

pytestmark = pytest.mark.gpu


def low_rank(count, rows, cols, rank, kind, seed, exact=False):
    """Products of thin matrices; exact: rows (or columns, of tall ones) that are the same, so that no rounding gives a rank."""
    g = gen_of(seed)
    if exact:
        short, long = min(rows, cols), max(rows, cols)
        x = torch.randn(count, rank, long, generator=g, device=DEV)[:, torch.arange(short, device=DEV) % rank]
        x = x if rows <= cols else x.transpose(1, 2)
        return x.contiguous().to(DT[kind])
    x = torch.bmm(torch.randn(count, rows, rank, generator=g, device=DEV), torch.randn(count, rank, cols, generator=g, device=DEV))
    return x.to(DT[kind])


THIN = [(1, 8, 256, 4), (2, 1000, 32, 16), (1, 64, 700, 20), (3, 500, 30, 1), (1, 32, 200, 4), (2, 8, 16, 1), (1, 3001, 47, 47), (1, 1, 900, 1)]


def verify_steps(g, o, kind, steps, coef):
    """As verify, and for what 64 bits leave: step_errors of rows that are the same is that of fp32 products, which keep them the
    same to the bit and so have nothing in the directions that are missing. Products that do not take all rows alike have
    sqrt(K) 2^-53 of the norm there after a step, K up to 3001 terms, and every later step multiplies it by a: sqrt(3001) 2^-53
    (a + a^2 + ... ) < 2^-53 2^5.8 a^steps a / (a - 1) < 2^-46 a^steps for a >= 1.875. In any case no singular value leaves
    the polynomial's range, 1.23 for these, but for 4 roundings of the result."""
    want, most = step_errors(g, DT[kind], steps=steps, coef=coef)
    rounding = off(want.to(o.dtype), want)
    got = off(o, want)
    bound = 1.1 * (rounding.square() + (most + 2.0 ** -46 * coef[0] ** steps).square()).sqrt()
    say("error", got.max().item(), "of", bound.max().item())
    assert torch.isfinite(o).all() and (got <= bound).all(), "%.3g of the bound" % (got / bound).max()
    x = o.double() if o.shape[1] <= o.shape[2] else o.double().transpose(1, 2).contiguous()
    largest = torch.linalg.eigvalsh(torch.bmm(x, x.transpose(1, 2).contiguous()).cpu()).amax(1).clamp(min=0).sqrt()
    assert (largest <= 1.23 + 4 * torch.finfo(o.dtype).eps).all(), largest.max()


@pytest.mark.parametrize("coef", [NS, (2.0, -1.5, 0.5), (1.875, -1.25, 0.375)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("exact", [False, True])
@pytest.mark.parametrize("count,rows,cols,rank", THIN)
def test_many_steps_of_thin_matrices(count, rows, cols, rank, exact, kind, coef):
    """What rounding makes of eigenvalues that are 0 must neither grow out of the range nor into the result."""
    g = low_rank(count, rows, cols, rank, kind, rows + rank, exact)
    for steps in (6, 8, 9, 12, 16, 17, 20, 25, 32):
        say("steps", steps, coef, count, rows, cols, "rank", rank, exact, kind)
        verify_steps(g, orthogonalize(g, kind, steps=steps, coefficients=coef), kind, steps, coef)


@pytest.mark.parametrize("count,rows,cols,rank", THIN)
def test_twelve_steps_of_thin_matrices(count, rows, cols, rank):
    """Two runs of 6 steps: each multiplies the rounding of Gram's matrix, 2^-53, by 11.9^6 = 2^21.4 at most, and the second what
    the first left by 3.4445^6 = 2^10.7: 2^-21 in all, and 2^-24 for the result's own rounding."""
    for exact in (False, True):
        g = low_rank(count, rows, cols, rank, "f32", rows, exact)
        got = off(orthogonalize(g, "f32", steps=12), newton_schulz(g, steps=12))
        say("error", got.max().item())
        assert (got <= 2.0 ** -21 + 2.0 ** -24).all()


def test_long_stack_of_many_steps():
    """More matrices than X is kept of at a time; a matrix's bits do not depend on the stack."""
    count, rows, cols = 700, 32, 2000
    assert count * rows * cols * 8 > 256 << 20
    g = matrices(count, rows, cols, "f32", seed=8, rank=2)
    ws = workspace("f32", count, rows, cols)
    o = torch.full_like(g, 5.0)
    N.moe_orthogonalize(g, o, ws, steps=11)
    verify(g, o, "f32", steps=11)
    for i in (0, 523, 524, 699):
        assert torch.equal(orthogonalize(g[i].clone(), "f32", steps=11), o[i])


@pytest.mark.parametrize("p,master", [("f32", False), ("bf16", True), ("bf16", False)])
@pytest.mark.parametrize("steps", [8, 12, 20])
def test_muon_of_thin_matrices_by_many_steps(steps, p, master):
    s = Step([(3, 8, 256), (2, 300, 30), (1, 64, 500), (700, 9)], p, master=master)
    for t, m in zip(s.g, s.m):  # of low rank, the momentum too
        for x in (t, m):
            z = (1, *x.shape) if x.dim() == 2 else tuple(x.shape)
            x.copy_(low_rank(*z, 2, "f32", z[1]).reshape(x.shape) * 1e-3)
    lr, mu, wd = 0.02, 0.9, 0.1
    want = []
    for i, t in enumerate(s.p):
        z = (1, *t.shape) if t.dim() == 2 else tuple(t.shape)
        u = s.g[i].double() + mu * (mu * s.m[i].double() + s.g[i].double())
        o, e = step_errors(u.reshape(z).float(), DT[p], steps=steps)
        old = (s.master[i] if master else t).double().reshape(z)
        size = lr * 0.2 * math.sqrt(max(z[1:]))
        want.append((old * (1 - lr * wd) - size * o, size * e * o.square().sum((1, 2)).sqrt(), 2.0 ** -22 * (old.abs() + (size * o).abs())))
    s.run(lr, mu, True, wd, steps=steps)
    for i, (new, far, near) in enumerate(want):
        got = (s.master[i] if master else s.p[i]).double().reshape(new.shape)
        half = 2.0 ** -8 if p == "bf16" and not master else 0.0
        d = ((got - new).abs() - near - half * new.abs() * 1.01).clamp(min=0).square().sum((1, 2)).sqrt()
        assert torch.isfinite(got).all() and (d <= far).all(), "tensor %d: %.3g of the bound" % (i, (d / far).max())
