"""Orthogonalisation and Muon steps with step counts and polynomials other than the usual ones, for every kind of kernel, on the GPU."""
import math

import pytest
import torch

from expert_ffn_layer_amd import native as N

from _gpu import say
from _muon import NS, newton_schulz, off, plain_steps, step_errors
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


def largest(o):
    """Each matrix's largest singular value."""
    x = o.double() if o.shape[1] <= o.shape[2] else o.double().transpose(1, 2).contiguous()
    return torch.linalg.eigvalsh(torch.bmm(x, x.transpose(1, 2).contiguous()).cpu()).amax(1).clamp(min=0).sqrt()


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
    assert (largest(o) <= 1.23 + 4 * torch.finfo(o.dtype).eps).all()


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


# A size for every kind of kernel: in 64 bits; one workgroup a matrix; Gram's matrix by parts of the reduction; products of 128 x 128
# tiles; of 256 x 256 tiles in every form, with rows that do and do not begin on 16 bytes.
KINDS = [(3, 40, 700), (2, 900, 30), (2, 100, 200), (3, 255, 127), (1, 300, 4000), (1, 2501, 130), (2, 640, 700), (1, 771, 650), (19, 1021, 1100), (19, 1100, 1024)]
FEW = [(NS, 1), (NS, 2), (NS, 8), ((1.5, -0.5, 0.0), 12), ((2.0, -1.5, 0.5), 10), ((1.0, 0.0, 0.0), 2), ((0.5, 0.0, 0.0), 3)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("z", KINDS)
def test_other_steps_and_polynomials(z, kind):
    g = matrices(*z, kind, seed=z[1])
    for coef, steps in FEW:
        say(z, coef, steps, kind)
        verify(g, orthogonalize(g, kind, steps=steps, coefficients=coef), kind, steps=steps, coef=coef)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("z", KINDS)
def test_low_rank(z, kind):
    """With what rounding leaves in the other directions: enlarged by every step, it must stay in the polynomial's range, whose end
    the steps' own rounding may pass by the 2% that the interface gives it. How far a result is off is known for few steps
    only: once the singular values are between 0.7 and 1.23 a step multiplies differences by |3.4445 - 14.325 s^2 + 10.1575 s^4|,
    1.6 inside and 4 at the end, so that two computations that round alike but not the same, 2^-12 apart, are 1 apart after
    some 12 to 18 more steps, and neither's error bounds the other's."""
    for rank in (1, 5):
        g = low_rank(*z, rank, kind, seed=rank)
        for steps in (5, 8, 10):
            say(z, "rank", rank, steps, kind)
            verify(g, orthogonalize(g, kind, steps=steps), kind, steps=steps)
        for steps in (16, 32) if z[0] < 19 else ():
            o = orthogonalize(g, kind, steps=steps)
            assert torch.isfinite(o).all() and (largest(o) <= 1.23 * 1.02).all(), steps


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("z", KINDS)
def test_a_matrix_that_is_not_finite_is_alone(z, kind):
    g = matrices(max(z[0], 3), *z[1:], kind)
    a = orthogonalize(g, kind)
    for bad in (math.nan, math.inf, -math.inf):
        x = g.clone()
        x[1, z[1] - 1, z[2] - 1] = bad
        for steps in (5, 1, 10):
            o = orthogonalize(x, kind, steps=steps)
            want = a if steps == 5 else orthogonalize(g, kind, steps=steps)
            assert o[1].isnan().all() and torch.equal(o[0], want[0]) and torch.equal(o[2:], want[2:]), (bad, steps)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("z", KINDS)
def test_scale_of_the_input_does_not_matter(z, kind):
    g = matrices(max(z[0], 2), *z[1:], kind)
    for steps in (5, 10):
        a = orthogonalize(g, kind, eps=0.0, steps=steps)
        for e in (-100, -60, 60, 100):
            assert torch.equal(orthogonalize(g * 2.0 ** e, kind, eps=0.0, steps=steps), a), (e, steps)
    zeros = torch.zeros_like(g)
    zeros[1] = g[1]
    for eps, steps in ((0.0, 5), (1e-7, 5), (0.0, 10)):
        o = orthogonalize(zeros, kind, eps=eps, steps=steps)
        assert (o[0] == 0).all() and torch.equal(o[1], orthogonalize(g, kind, eps=eps, steps=steps)[1])
    eps = float(g[0].double().square().sum().sqrt())  # halves the first matrix's singular values
    verify(g, orthogonalize(g, kind, eps=eps), kind, eps=eps)


@pytest.mark.parametrize("p,g,master", [("f32", "f32", False), ("bf16", "bf16", False), ("bf16", "f32", True)])
@pytest.mark.parametrize("steps", [1, 5, 8])
@pytest.mark.parametrize("tall", [False, True])
def test_step_by_other_numbers_of_steps(steps, p, g, master, tall):
    sizes = [(n, c, r) if tall else (n, r, c) for n, r, c in ((3, 40, 700), (2, 100, 200), (1, 300, 4000), (2, 640, 701), (19, 1024, 1100))]
    s = Step(sizes, p, g, master, seed=steps)
    want = s.want(0.02, 0.9, True, 0.1)
    for i, t in enumerate(s.p):  # with this many steps in place of the usual
        u = s.g[i].double() + 0.9 * want[i][3].reshape(t.shape)
        o, e = step_errors(u, DT[p], steps=steps)
        old = (s.master[i] if master else t).double()
        size = 0.02 * 0.2 * math.sqrt(max(t.shape[1:]))
        want[i] = (old * (1 - 0.02 * 0.1) - size * o, size * e * o.square().sum((1, 2)).sqrt(), 2.0 ** -22 * (old.abs() + (size * o).abs()), *want[i][3:])
    s.run(0.02, 0.9, True, 0.1, steps=steps)
    s.verify(want)


def pair_steps(g, steps=5, coef=NS, eps=1e-7):
    """The steps with the operands of fp32 matrices' products as pairs of fp16, whose lower halves are not multiplied with each
    other, and nothing else rounded."""
    a, b, c = coef
    S = 4096.0

    def pair(t):
        hi = t.half().double()
        return hi, (t - hi).half().double()

    def product(p, q):
        (ph, pl), (qh, ql) = pair(p), pair(q)
        return torch.bmm(ph + pl, qh + ql) - torch.bmm(pl, ql)
    x = g.double()
    x = x * (S / (x.square().sum((1, 2), keepdim=True).sqrt() + eps))
    wide = x.shape[1] <= x.shape[2]
    x = x if wide else x.transpose(1, 2).contiguous()
    one = torch.eye(x.shape[1], dtype=torch.float64, device=x.device)
    for _ in range(steps):
        A = product(x, x.transpose(1, 2).contiguous()) / S
        d = torch.diag_embed(torch.diagonal(A, dim1=1, dim2=2))
        C = b * A + c * (product(A - d, A - d) + torch.bmm(d, A) + torch.bmm(A, d) - torch.bmm(d, d)) / S + a * S * one
        x = product(C, x) / S
    x = x / S
    return x if wide else x.transpose(1, 2).contiguous()


@pytest.mark.parametrize("rank", [0, 16, 1])
@pytest.mark.parametrize("z", [z for z in KINDS if min(z[1:]) > 64])
def test_error_of_fp32(z, rank):
    """That of the operands, which pair_steps has, twice for single operands that go the other way, and that of fp32 sums, which
    fp32 products have: three sums of the same length in place of one, sqrt(3) < 2 times."""
    g = gen_of(rank)
    x = torch.randn(z, generator=g, device=DEV) if rank == 0 else low_rank(*z, rank, "f32", rank) + (0.0 if rank == 1 else torch.randn(z, generator=g, device=DEV))
    want = newton_schulz(x)
    got, plain, pairs = off(orthogonalize(x, "f32"), want), off(plain_steps(x), want), off(pair_steps(x), want)
    say(z, rank, "error", got.max().item(), "fp32 products", plain.max().item(), "pairs", pairs.max().item())
    assert (got <= 2 * plain + 2 * pairs + 2.0 ** -24).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_many_steps_in_graphs_and_in_bounds(kind):
    """Thin matrices, whose X passes through the workspace: two graphs that share one, other bytes in it, and what lies behind."""
    for z in ((3, 40, 700), (2, 900, 31), (5, 7, 9)):
        g = matrices(*z, kind, seed=z[1])
        n, need = g.numel(), N.moe_orthogonalize_workspace_size(kind, *z)
        ws = torch.full((need + 4096,), 0xAB, dtype=torch.uint8, device=DEV)
        outs = [torch.full((n + 64,), 5.0, dtype=DT[kind], device=DEV) for _ in range(2)]
        orthogonalize(g, kind, steps=12)
        torch.cuda.synchronize()
        graphs = [torch.cuda.CUDAGraph() for _ in outs]
        for graph, o in zip(graphs, outs):
            with torch.cuda.graph(graph):
                N.moe_orthogonalize(g, o[:n].reshape(z), ws[:need], steps=12)
        for i in range(3):
            g.copy_(torch.randn(z, device=DEV))
            ws[:need].fill_(0x11 * i)
            for graph in graphs:
                graph.replay()
            want = orthogonalize(g, kind, steps=12)
            torch.cuda.synchronize()
            assert all(torch.equal(o[:n].reshape(z), want) for o in outs), "replay %d" % i
        assert all((o[n:] == 5.0).all() for o in outs) and (ws[need:] == 0xAB).all()
