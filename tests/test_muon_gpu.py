"""Orthogonalisation by Newton-Schulz products and the Muon step on the GPU against their 64-bit definitions."""
import math

import pytest
import torch

from expert_ffn_layer_amd import native as N

from _gpu import say
from _muon import NS, newton_schulz, off, step_errors

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def gen_of(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def matrices(count, rows, cols, kind, seed=1, rank=4, size=1.0):
    """A few strong directions over noise."""
    g = gen_of(seed)
    r = min(rank, rows, cols)
    x = torch.bmm(torch.randn(count, rows, r, generator=g, device=DEV), torch.randn(count, r, cols, generator=g, device=DEV))
    return ((x + torch.randn(count, rows, cols, generator=g, device=DEV)) * size).to(DT[kind])


def workspace(kind, *size):
    return torch.full((N.moe_orthogonalize_workspace_size(kind, *size),), 0xFF, dtype=torch.uint8, device=DEV)


def orthogonalize(g, kind, **kw):
    o = torch.full_like(g, 123.0)
    size = g.shape if g.dim() == 3 else (1, *g.shape)
    N.moe_orthogonalize(g, o, workspace(kind, *size), **kw)
    return o


def verify(g, o, kind, **kw):
    want, most = step_errors(g, DT[kind], **kw)
    rounding = off(want.to(o.dtype), want)
    got = off(o, want)
    bound = 1.1 * (rounding.square() + most.square()).sqrt()
    worst = (got / bound.clamp(min=1e-30)).max().item()
    say("error", got.max().item(), "of", bound.max().item())
    assert torch.isfinite(o).all() and worst <= 1.0, "%.3g of the bound" % worst


SIZES = [(1, 1, 1), (3, 1, 7), (2, 9, 1), (5, 8, 8), (2, 64, 64), (3, 65, 63), (2, 63, 65), (1, 200, 130), (3, 130, 200), (2, 257, 64),
         (1, 64, 700), (1, 513, 384), (2, 300, 520), (1, 1000, 257)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("count,rows,cols", SIZES)
def test_sizes(count, rows, cols, kind):
    say("orthogonalize", count, rows, cols, kind)
    g = matrices(count, rows, cols, kind, seed=rows)
    verify(g, orthogonalize(g, kind), kind)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_many_tiles(kind):
    for count, rows, cols in ((2, 1100, 900), (3, 640, 1664)):
        say("orthogonalize", count, rows, cols, kind)
        g = matrices(count, rows, cols, kind, seed=7, rank=16)
        verify(g, orthogonalize(g, kind), kind)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("count,rows,cols", [(1, 70, 900), (2, 79, 4042), (1, 6100, 150), (1, 400, 9000), (5, 380, 1100)])
def test_few_tiles_with_a_long_reduction(count, rows, cols, kind):
    say("orthogonalize", count, rows, cols, kind)
    g = matrices(count, rows, cols, kind, seed=rows)
    o = orthogonalize(g, kind)
    verify(g, o, kind)
    assert torch.equal(o, orthogonalize(g, kind))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_long_stack(kind):
    """More matrices than are worked on at a time."""
    g = matrices(2500, 8, 11, kind, seed=3, rank=2)
    o = orthogonalize(g, kind)
    verify(g, o, kind)
    one = orthogonalize(g[1300].clone(), kind)
    assert torch.equal(one, o[1300])  # a matrix's bits do not depend on the stack


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_low_rank(kind):
    """As an expert's gradient that few tokens reach: what is 0 stays near 0 although steps enlarge it 485 times."""
    for rank, size in ((1, (96, 160)), (3, (300, 128)), (2, (128, 128))):
        g = gen_of(rank)
        x = torch.bmm(torch.randn(2, size[0], rank, generator=g, device=DEV), torch.randn(2, rank, size[1], generator=g, device=DEV))
        x = x.to(DT[kind])
        say("rank", rank, size, kind)
        verify(x, orthogonalize(x, kind), kind)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_scale_of_the_input_does_not_matter(kind):
    g = matrices(2, 70, 90, kind)
    a = orthogonalize(g, kind, eps=0.0)
    for e in (-100, -60, 60, 100):
        assert torch.equal(orthogonalize(g * 2.0 ** e, kind, eps=0.0), a)
    z = torch.zeros_like(g)
    z[1] = g[1]
    for eps in (0.0, 1e-7):
        o = orthogonalize(z, kind, eps=eps)
        assert (o[0] == 0).all() and torch.equal(o[1], orthogonalize(g, kind, eps=eps)[1])
    big = orthogonalize(g, kind, eps=float(g[0].double().square().sum().sqrt()))  # halves the first matrix's singular values
    want = newton_schulz(g, eps=float(g[0].double().square().sum().sqrt()))
    assert off(big, want).max() < 0.01


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_other_steps_and_polynomials(kind):
    g = matrices(2, 80, 112, kind)
    for coef, steps in ((NS, 1), (NS, 8), ((1.5, -0.5, 0.0), 12), ((2.0, -1.5, 0.5), 10), ((1.0, 0.0, 0.0), 2), ((0.5, 0.0, 0.0), 3)):
        say(coef, steps, kind)
        verify(g, orthogonalize(g, kind, steps=steps, coefficients=coef), kind, steps=steps, coef=coef)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_matrix_that_is_not_finite_is_alone(kind, bad):
    g = matrices(3, 100, 70, kind)
    a = orthogonalize(g, kind)
    g[1, 99, 69] = bad
    o = orthogonalize(g, kind)
    assert o[1].isnan().all() and torch.equal(o[0], a[0]) and torch.equal(o[2], a[2])


def test_empty_stacks():
    for size in ((0, 5, 5), (3, 0, 5), (3, 5, 0)):
        g = torch.empty(size, device=DEV)
        assert N.moe_orthogonalize_workspace_size("f32", *size) == 0
        N.moe_orthogonalize(g, g.clone(), torch.empty(0, dtype=torch.uint8, device=DEV))


class Step:
    def __init__(self, sizes, p="bf16", g=None, master=False, seed=1):
        gen = gen_of(seed)
        g = g or p
        w = [torch.randn(z, generator=gen, device=DEV) * 0.02 for z in sizes]
        self.p = [t.to(DT[p]) for t in w]
        self.master = w if master else None
        self.g = [matrices(*(z if len(z) == 3 else (1, *z)), g, seed + 1 + i, size=1e-3).reshape(z) for i, z in enumerate(sizes)]
        self.m = [matrices(*(z if len(z) == 3 else (1, *z)), "f32", seed + 50 + i, size=1e-2).reshape(z) for i, z in enumerate(sizes)]
        self.kind = p
        self.table = N.muon_tensors(self.p, self.g, self.m, self.master)
        self.ws = torch.full((N.moe_muon_workspace_size(self.table),), 0xFF, dtype=torch.uint8, device=DEV)

    def arrays(self):
        return self.p + self.m + (self.master or [])

    def want(self, lr, momentum, nesterov, wd, gs=1.0):
        """(p, bound, m, bound) of each tensor, from the present values."""
        out = []
        for i, p in enumerate(self.p):
            z = p.shape if p.dim() == 3 else (1, *p.shape)
            g, m = self.g[i].double().reshape(z) * gs, self.m[i].double().reshape(z)
            m1 = momentum * m + g
            # three roundings of fp32, and one more where g is scaled
            tm = 2.0 ** -22 * ((momentum * m).abs() + g.abs())
            u = g + momentum * m1 if nesterov else m1
            o, e = step_errors(u, DT[self.kind])
            old = (self.master[i] if self.master else p).double().reshape(z)
            s = lr * 0.2 * math.sqrt(max(z[1:]))
            new = old * (1 - lr * wd) - s * o
            # O's error, as that of its norm, and four roundings of fp32
            norm = o.square().sum((1, 2)).sqrt()
            out.append((new, s * e * norm, 2.0 ** -22 * (old.abs() + (s * o).abs()), m1, tm))
        return out

    def verify(self, want):
        for i, (new, far, near, m1, tm) in enumerate(want):
            z = new.shape
            assert ((self.m[i].reshape(z).double() - m1).abs() <= tm).all(), "momentum %d" % i
            w = (self.master[i] if self.master else self.p[i]).reshape(z).double()
            half = 0.0 if self.master or self.kind == "f32" else 2.0 ** -8
            d = ((w - new).abs() - near - half * new.abs() * 1.01).clamp(min=0).square().sum((1, 2)).sqrt()
            assert (d <= far).all(), "tensor %d: %.3g of the bound" % (i, (d / far).max())
            if self.master:
                assert torch.equal(self.p[i], self.master[i].to(torch.bfloat16))

    def run(self, lr=0.02, momentum=0.9, nesterov=True, wd=0.1, **kw):
        N.moe_muon(self.table, self.ws, lr=lr, momentum=momentum, nesterov=nesterov, weight_decay=wd, **kw)


STACKS = [(3, 64, 128), (3, 128, 64), (2, 128, 64), (100, 37), (1, 37, 100), (1, 1), (5, 3, 200), (0, 64, 128), (2, 130, 130)]


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("p,g,master", [("f32", "f32", False), ("bf16", "bf16", False), ("bf16", "f32", True), ("bf16", "bf16", True),
                                        ("f32", "bf16", False)])
def test_step(p, g, master, nesterov):
    say("muon", p, g, master, nesterov)
    s = Step(STACKS, p, g, master)
    for lr, momentum, wd in ((0.02, 0.9, 0.1), (0.3, 0.0, 0.0)):
        want = s.want(lr, momentum, nesterov, wd)
        s.run(lr, momentum, nesterov, wd)
        s.verify(want)


def test_device_values():
    s = Step(STACKS[:4])
    lr, gs = torch.tensor([0.05], device=DEV), torch.tensor([0.25], device=DEV)
    want = s.want(0.05, 0.9, True, 0.1, 0.25)
    s.run(lr=7.0, lr_dev=lr, grad_scale=gs)
    s.verify(want)


def test_more_stacks_than_a_launch_holds():
    s = Step([(1, 24, 40 if i % 2 else 24) for i in range(95)], "f32")
    want = s.want(0.02, 0.9, True, 0.1)
    s.run()
    s.verify(want)


def test_same_bits_on_every_run_and_stream():
    a, b = Step(STACKS, master=True), Step(STACKS, master=True)
    a.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    b.ws.fill_(0x55)
    torch.cuda.synchronize()
    b.run(stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a.arrays(), b.arrays()))


def test_captured_step():
    """Replays follow the device values and gradients, with eager steps of another table between them."""
    a, b, c = (Step(STACKS, master=True) for _ in range(3))
    lr = torch.tensor([0.02], device=DEV)
    start = [t.clone() for t in a.arrays()]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        a.run(lr_dev=lr)
    torch.cuda.current_stream().wait_stream(stream)
    for t, z in zip(a.arrays(), start):
        t.copy_(z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run(lr_dev=lr)
    for i in range(4):
        lr.fill_(0.02 / (i + 1))
        for x, y in zip(a.g, b.g):
            x.mul_(-0.5)
            y.mul_(-0.5)
        graph.replay()
        c.run()
        b.run(lr=float(lr))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a.arrays(), b.arrays())), "replay %d" % i


KINDS_OF_WORK = [(3, 40, 700), (2, 100, 200), (1, 300, 4000), (2, 640, 700)]  # in 64 bits, one workgroup, shared reductions, products


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_captured_orthogonalize(kind):
    gs = [matrices(*z, kind, seed=i) for i, z in enumerate(KINDS_OF_WORK)]
    os, ws = [torch.empty_like(g) for g in gs], [workspace(kind, *z) for z in KINDS_OF_WORK]

    def all_of(os, ws):
        for g, o, w in zip(gs, os, ws):
            N.moe_orthogonalize(g, o, w)
    all_of(os, ws)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = [[torch.empty_like(g) for g in gs] for _ in graphs]
    for graph, o in zip(graphs, outs):  # two graphs that share workspaces, replayed one after the other
        with torch.cuda.graph(graph):
            all_of(o, ws)
    for i in range(4):
        for g in gs:
            g.copy_(torch.randn(g.shape, device=DEV))
        for graph in graphs:
            graph.replay()
        all_of(os, [workspace(kind, *z) for z in KINDS_OF_WORK])
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(x, y) for x, y in zip(o, os)), "replay %d" % i


def test_two_calls_at_once():
    """On two streams, with a workspace each."""
    for z in KINDS_OF_WORK:
        gs = [matrices(*z, "bf16", seed=i) for i in range(2)]
        want = [orthogonalize(g, "bf16") for g in gs]
        os, ws, streams = [torch.empty_like(g) for g in gs], [workspace("bf16", *z) for _ in gs], [torch.cuda.Stream() for _ in gs]
        torch.cuda.synchronize()
        for _ in range(5):
            for g, o, w, s in zip(gs, os, ws, streams):
                N.moe_orthogonalize(g, o, w, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(os, want)), z


@pytest.mark.parametrize("p,master", [("f32", False), ("bf16", True)])
def test_step_of_every_kind_of_work(p, master):
    """Matrices of each kernel's sizes in one step, both ways round and at lengths that are not multiples of 4 or 8."""
    s = Step([(2, 33, 1001), (1, 1001, 33), (2, 127, 255), (1, 255, 127), (1, 129, 3001), (1, 2051, 130), (1, 515, 770)], p, master=master)
    for lr, momentum, nesterov in ((0.02, 0.95, True), (0.1, 0.5, False)):
        want = s.want(lr, momentum, nesterov, 0.1)
        s.run(lr, momentum, nesterov, 0.1)
        s.verify(want)


def test_nothing_is_written_past_the_end():
    for kind in ("f32", "bf16"):
        for z in ((3, 7, 9), (2, 101, 203), (1, 301, 333), (1, 130, 2501)):
            n = z[0] * z[1] * z[2]
            need = N.moe_orthogonalize_workspace_size(kind, *z)
            buf = torch.full((n + 64,), 5.0, dtype=DT[kind], device=DEV)
            ws = torch.full((need + 4096,), 0xAB, dtype=torch.uint8, device=DEV)
            N.moe_orthogonalize(matrices(*z, kind), buf[:n].reshape(z), ws[:need])
            assert (buf[n:] == 5.0).all() and (ws[need:] == 0xAB).all(), (kind, z)
