"""The training operators on the GPU against their 64-bit definitions: the gated block that keeps its
pre-activations, its gradient, the combine's gradient, AdamW, and a training step of them together."""
import math

import pytest
import torch

from expert_ffn_layer_amd import native as N
from expert_ffn_layer_amd.layer import TrainableLayer
from inputgen import layers as L

from _gpu import say
from _train import A, DT, F, backward, check, forward, half_step, layout

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
SENTINEL = 12345.0


def gen_of(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)


class Block:
    """Inputs and outputs of the block for rows grouped as `counts`, in T*k >= sum(counts) row slots."""

    def __init__(self, counts, H, I, act, seed=1, spare=3, gather=True, dense=False):
        self.counts, self.H, self.I, self.act, self.dtype = counts, H, I, act, DT[act]
        E, n = len(counts), sum(counts)
        self.k = 2 if E > 1 else 1
        self.T = (n + self.k - 1) // self.k + (0 if dense else spare)
        self.P, self.n, self.E = self.T * self.k, n, E
        gen = gen_of(seed)
        cpu = torch.Generator().manual_seed(seed)
        self.off, slot = layout(counts, self.T, cpu, DEV)
        self.slot = torch.full((self.P,), -7, dtype=torch.int32, device=DEV)
        self.slot[:n] = slot
        if not gather:
            self.slot = None
        self.x = normal(gen, (self.T if gather else self.P, H), self.dtype)
        self.w = {"gate": normal(gen, (E, H, I), self.dtype, H ** -0.5), "up": normal(gen, (E, H, I), self.dtype, H ** -0.5),
                  "down": normal(gen, (E, I, H), self.dtype, I ** -0.5)}
        self.g, self.u = normal(gen, (self.P, I), self.dtype, 2.0), normal(gen, (self.P, I), self.dtype)
        self.dy = normal(gen, (self.P, H), self.dtype)
        if dense:
            self.off = self.slot = None
        self.shape = N.make_shape(self.T, H, E, self.k, I, act=act, w_routed=act)
        self.ws = torch.full((N.moe_train_workspace_size(self.shape),), 0xFF, dtype=torch.uint8, device=DEV)

    def rows(self, e):
        a = sum(self.counts[:e])
        return a, a + self.counts[e]

    def xrows(self, a, b):
        return (self.x[a:b] if self.slot is None else self.x[self.slot[a:b].long()]).double()

    def empty(self, *shape):
        return torch.full(shape, SENTINEL, dtype=self.dtype, device=DEV)

    def forward(self, keep=True):
        g, u = (self.empty(self.P, self.I) if keep else None for _ in range(2))
        y = self.empty(self.P, self.H)
        N.moe_gated_ffn(self.shape, self.x, self.off, self.slot, self.w, g, u, y, self.ws)
        return {"g": g, "u": u, "y": y}

    def backward(self, dx=True, grads=True):
        out = {"dx": self.empty(self.P, self.H) if dx else None}
        gr = {n: torch.full_like(t, SENTINEL) for n, t in self.w.items()} if grads else None
        N.moe_gated_ffn_backward(self.shape, self.x, self.off, self.slot, self.w, self.g, self.u, self.dy, out["dx"], gr, self.ws)
        return out | ({"d" + n: t for n, t in gr.items()} if grads else {})

    def want(self, e, which):
        a, b = self.rows(e)
        w = [self.w[n][e].double() for n in ("gate", "up", "down")]
        if which == "forward":
            return forward(self.xrows(a, b), *w, self.dtype)
        return backward(self.xrows(a, b), *w, self.g[a:b].double(), self.u[a:b].double(), self.dy[a:b].double(), self.dtype)

    def verify(self, got, which, experts=None):
        worst = 0.0
        for e in range(self.E) if experts is None else experts:
            a, b = self.rows(e)
            for name, (value, bound) in self.want(e, which).items():
                if got.get(name) is None:
                    continue
                part = got[name][e] if name in ("dgate", "dup", "ddown") else got[name][a:b]
                worst = max(worst, check("%s of expert %d" % (name, e), part, value, bound))
        for name in ("g", "u", "y", "dx"):
            if got.get(name) is not None:
                assert (got[name][self.n:] == SENTINEL).all(), "%s: rows past the last group were written" % name
        return worst


LAYOUTS = {
    "one-row": [1],
    "ragged": [0, 1, 63, 64, 0, 65, 128, 2, 257, 0],
    "many-small": [3, 0, 1, 5, 2, 0, 0, 7, 1, 4, 2, 9, 1, 0, 3, 17] * 5,
    "large-group": [700, 5],
}
SIZES = {"one-row": (128, 128), "ragged": (256, 384), "many-small": (384, 128), "large-group": (640, 256)}


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("name", LAYOUTS)
def test_block_and_gradient(name, act):
    H, I = SIZES[name]
    b = Block(LAYOUTS[name], H, I, act, seed=11)
    say("block", name, act, b.T, b.k, H, I)
    f = b.verify(b.forward(), "forward")
    say("forward worst", f)
    r = b.verify(b.backward(), "backward")
    say("backward worst", r)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 129, 1000])
def test_dense_block(rows, act):
    """E = 1 without offsets or gather, H and I odd multiples of 128."""
    b = Block([rows], 896, 640, act, seed=5, gather=False, dense=True)
    say("dense", rows, act)
    b.verify(b.forward(), "forward")
    b.verify(b.backward(), "backward")


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_wide_sizes(act):
    """The benchmark widths of the V3 layer, few rows; more experts than lanes of a wave on the small one."""
    b = Block([5, 0, 130], 7168, 2048, act, seed=6)
    say("wide", act)
    b.verify(b.forward(), "forward")
    b.verify(b.backward(), "backward")
    c = Block([i % 3 for i in range(200)], 128, 128, act, seed=7)
    c.verify(c.forward(), "forward", range(0, 200, 7))
    c.verify(c.backward(), "backward", range(0, 200, 7))


# Rows per group, H and I that take every tile shape of every product in bf16 (256 x 256, 128 x 128, 64 x 256 and
# 64 x 128, the last two also with the weights streamed) and both of fp32, with H and I odd multiples of 128 and
# groups that end inside and at the end of a tile
TILES = {
    "thin": ([2, 5, 2, 6, 8, 4, 4, 2, 0, 3, 9, 1], 1664, 2688),
    "thin-many": ([1, 3, 19, 9, 16, 4, 2, 66, 1, 3, 20, 13, 4, 0, 2, 1, 10, 2, 0, 5], 2176, 2176),
    "mixed": ([64, 149, 0, 1200, 589, 256, 405, 1200, 736, 129, 173, 412], 384, 384),
    "many-rows": ([1125, 452, 204, 0, 831, 398, 53, 75, 2400, 512, 257, 87, 2400, 476, 128, 690, 1, 255, 968, 368], 384, 384),
    "wide": ([978, 408, 0, 598, 1281, 291, 242, 298, 616], 1664, 384),
    "uneven": ([90, 67, 35, 80, 27, 0, 58, 143, 107, 68, 150, 0, 15, 10, 24, 150, 12, 44, 70, 102], 1664, 1152),
    "two-rows": ([1, 1], 7040, 3968),
    "deep": ([86, 282, 96, 18, 33, 300, 300, 42, 131, 40, 58, 173, 1, 14, 0, 274, 15, 51, 129, 222], 384, 2688),
}


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("name", TILES)
def test_tile_shapes(name, act):
    counts, H, I = TILES[name]
    b = Block(counts, H, I, act, seed=21)
    say("tiles", name, act, b.T, b.k, H, I)
    say("forward worst", b.verify(b.forward(), "forward"))
    say("backward worst", b.verify(b.backward(), "backward"))


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_a_row_does_not_depend_on_the_others(act):
    """The first rows of each group alone give the bits they give among all, in other tile shapes."""
    counts, H, I = [1300, 0, 2047, 600], 2432, 640
    b = Block(counts, H, I, act, seed=22, gather=False)
    say("row alone", act)
    full = b.forward() | b.backward(grads=False)
    few = [33, 0, 70, 1]
    c = Block(few, H, I, act, seed=23, gather=False)
    c.w = b.w
    pick = torch.cat([torch.arange(b.rows(e)[0], b.rows(e)[0] + n, device=DEV) for e, n in enumerate(few)])
    for name in ("x", "g", "u", "dy"):
        getattr(c, name)[:c.n] = getattr(b, name)[pick]
    part = c.forward() | c.backward(grads=False)
    for name in ("g", "u", "y", "dx"):
        assert torch.equal(part[name][:c.n], full[name][pick]), name


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_rows_in_order_and_partial_outputs(act):
    """slot_token NULL reads x by row; pre-activations, dx and the weight gradients may be left out."""
    b = Block([40, 0, 90], 256, 128, act, seed=8, gather=False)
    say("partial", act)
    full = b.forward()
    b.verify(full, "forward")
    assert torch.equal(b.forward(keep=False)["y"], full["y"])
    back = b.backward()
    b.verify(back, "backward")
    assert torch.equal(b.backward(grads=False)["dx"], back["dx"])
    only = b.backward(dx=False)
    assert all(torch.equal(only[n], back[n]) for n in ("dgate", "dup", "ddown"))


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_other_rows_do_not_reach_a_group(act):
    """NaN and infinity in rows past the last group, in another group's rows and in unused tokens stay there."""
    b = Block([70, 33, 50], 256, 256, act, seed=9)
    say("poison", act)
    b.slot[:b.n] = torch.arange(b.n, dtype=torch.int32, device=DEV) % (b.T - 2)  # two tokens unused
    first, last = b.rows(1)
    b.slot[first:last] = b.T - 1  # expert 1 reads one poisoned token
    b.x[b.T - 2:] = float("nan")
    for t in (b.g, b.u, b.dy):
        t[b.n:] = float("nan")
        t[first:last] = float("inf")
    f, r = b.forward(), b.backward()
    b.verify(f, "forward", [0, 2])
    b.verify(r, "backward", [0, 2])
    assert torch.isnan(f["y"][first:last].float()).all()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_tokens_outside_read_zeros_and_bad_offsets_stay_inside(act):
    b = Block([20, 30], 256, 128, act, seed=10)
    say("bad indices", act)
    b.slot[3], b.slot[25] = -1, b.T
    got = b.forward()
    for r in (3, 25):
        assert (got["y"][r] == 0).all() and (got["g"][r] == 0).all()
    b.slot[3], b.slot[25] = 0, 0
    # offsets that run backwards or past the rows: clamped, a group that ends before it begins is empty
    b.off = torch.tensor([0, 1 << 30, -5], dtype=torch.int32, device=DEV)
    b.slot = torch.zeros(b.P, dtype=torch.int32, device=DEV)
    out = b.forward()
    b.counts, b.E, b.n = [b.P], 1, b.P
    b.verify(out, "forward", [0])


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_no_tokens(act):
    """T = 0: nothing is written but the weight gradients, which are zero."""
    b = Block([0, 0], 128, 128, act, spare=0)
    say("empty", act)
    assert b.T == 0
    b.forward()
    out = b.backward()
    assert all((out[n] == 0).all() for n in ("dgate", "dup", "ddown"))


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_gradient_against_differences(act):
    """<dL/dw, d> of L = <y, c> against central differences of the 64-bit forward, for every input.
    The difference's own error is O(step^2); the gradient's is the operators' bound summed over |d|."""
    b = Block([9, 0, 23], 128, 128, act, seed=12)
    say("differences", act)
    out = b.forward()
    b.g, b.u = out["g"], out["u"]
    got = b.backward()
    un = half_step(b.dtype)
    gen = gen_of(13)
    for e in (0, 2):
        a, z = b.rows(e)
        x, c = b.xrows(a, z), b.dy[a:z].double()
        w = [b.w[n][e].double() for n in ("gate", "up", "down")]

        def loss(x, gate, up, down):
            g = x @ gate
            return ((g * torch.sigmoid(g) * (x @ up)) @ down * c).sum()
        for i, name in enumerate(("dx", "dgate", "dup", "ddown")):
            args = [x] + w
            d = torch.randn(args[i].shape, generator=gen, device=DEV, dtype=torch.float64) * args[i].std()
            step = 1e-4
            hi, lo = ([t + s * step * d if j == i else t for j, t in enumerate(args)] for s in (1, -1))
            diff = (loss(*hi) - loss(*lo)) / (2 * step)
            grad = got[name][a:z] if name == "dx" else got[name][e]
            slope = (grad.double() * d).sum()
            # g and u were rounded before the gradient read them: |d2L| of a rounding is at most about 3 of
            # them per factor of dg, du and h; all told 8 half steps of each product's magnitudes
            size = (grad.double().abs() * d.abs()).sum()
            assert (slope - diff).abs() <= 8 * un * size + 1e-6 * size, (name, e, slope.item(), diff.item())


@pytest.mark.slow
def test_rows_past_32_bit_offsets():
    """Row arrays of more than 2^31 elements (and 2^32 bytes): the last rows against the definition."""
    rows, H, I = 300_001, 7168, 128
    b = Block([rows], H, I, "bf16", seed=14, gather=False, dense=True)
    say("far rows", rows)
    assert rows * H > 1 << 31
    f = b.forward()
    r = b.backward(grads=False)
    a = rows - 40
    w = [b.w[n][0].double() for n in ("gate", "up", "down")]
    for name, (value, bound) in forward(b.x[a:].double(), *w, b.dtype).items():
        check(name, f[name][a:], value, bound)
    value, bound = backward(b.x[a:].double(), *w, b.g[a:].double(), b.u[a:].double(), b.dy[a:].double(), b.dtype)["dx"]
    check("dx", r["dx"][a:], value, bound)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_same_bits_on_every_run_streams_and_graphs(act):
    """Two streams at once with a workspace each, and a captured pass replayed between eager ones."""
    a, b = (Block([60, 0, 200, 31], 512, 256, act, seed=s) for s in (15, 16))
    say("streams", act)
    base = [(t.forward(), t.backward()) for t in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    again = []
    for _ in range(3):
        again = []
        for t, s in zip((a, b), streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                again.append((t.forward(), t.backward()))
        torch.cuda.synchronize()
        for x, y in zip(base, again):
            for p, q in zip(x, y):
                assert all(torch.equal(p[n], q[n]) for n in p)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out = (a.forward(), a.backward())
    for _ in range(4):
        for d in out:
            for t in d.values():
                t.fill_(SENTINEL)
        a.ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(base[0], out):
            assert all(torch.equal(p[n], q[n]) for n in p)
        b.forward()
        torch.cuda.synchronize()


# ------------------------------------------------------------------------------------------------
# combine

@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,k", [(1, 128, 1), (7, 384, 3), (65, 2560, 8), (33, 7168, 16)])
def test_combine_backward(T, H, k, act):
    say("combine backward", T, H, k, act)
    gen, dtype = gen_of(T + H), DT[act]
    P = T * k
    slot = torch.randperm(P, generator=gen, device=DEV).int()
    slot[torch.rand(P, generator=gen, device=DEV) < 0.2] = -1
    if P > 3:
        slot[1], slot[2] = P, -(1 << 31)
    slot = slot.reshape(T, k)
    w = torch.rand((T, k), generator=gen, device=DEV)
    dy, y = normal(gen, (T, H), dtype), normal(gen, (P, H), dtype)
    rows = torch.full((P, H), SENTINEL, dtype=dtype, device=DEV)
    dw = torch.full((T, k), SENTINEL, device=DEV)
    shape = N.make_shape(T, H, max(k, 2), k, 128, act=act, w_routed=act)
    N.moe_combine_backward(shape, dy, y, slot, w, rows, dw)
    ok = (slot >= 0) & (slot < P)
    assert (dw[~ok] == 0).all()
    t = torch.arange(T, device=DEV)[:, None].expand(T, k)[ok]
    s = slot[ok].long()
    a, b = dy[t].double(), y[s].double()
    check("dw", dw[ok], (a * b).sum(1), H * A * (a * b).abs().sum(1))
    want = torch.full((P, H), SENTINEL, dtype=torch.float64, device=DEV)
    want[s] = w[ok].double()[:, None] * a
    check("dy_perm", rows, want, half_step(dtype) * want.abs() + A * want.abs())
    # its rows against the combine itself: <combine(y), dy> = <y, dy_perm> = <w, dw>
    out = torch.empty((T, H), dtype=dtype, device=DEV)
    N.moe_combine(shape, y, slot, w, None, out)
    mags = (w[ok].double()[:, None] * (a * b).abs()).sum().item()
    left, right = (out.double() * dy.double()).sum().item(), (w.double() * dw.double()).sum().item()
    assert abs(left - right) <= (half_step(dtype) + (k + H + 2) * A) * mags


def test_combine_backward_keeps_nan_in_its_pair():
    gen = gen_of(3)
    T, H, k = 6, 256, 2
    slot = torch.arange(T * k, device=DEV, dtype=torch.int32).reshape(T, k)
    y, dy = normal(gen, (T * k, H), torch.bfloat16), normal(gen, (T, H), torch.bfloat16)
    y[3] = float("nan")
    rows, dw = torch.zeros_like(y), torch.zeros((T, k), device=DEV)
    shape = N.make_shape(T, H, 2, k, 128)
    N.moe_combine_backward(shape, dy, y, slot, torch.ones((T, k), device=DEV), rows, dw)
    assert torch.isnan(dw).sum() == 1 and torch.isnan(dw[1, 1])
    assert torch.isfinite(rows.float()).all()


# ------------------------------------------------------------------------------------------------
# AdamW

def dequantise(codes, scale):
    block = torch.arange(codes.numel(), device=DEV) // 256
    return codes.view(torch.float8_e4m3fn).double() * scale.double()[block]


def adam_case(sizes, p, g, master, state, seed, scale=1e-3):
    gen = gen_of(seed)
    c = {"p": [normal(gen, (n,), DT[p], 0.05) for n in sizes], "g": [normal(gen, (n,), DT[g], scale) for n in sizes],
         "master": None, "ms": None, "rs": None}
    if master:
        c["master"] = [t.float() + normal(gen, t.shape, torch.float32, 1e-5) for t in c["p"]]
    if state == "e4m3":
        blocks = [(n + 255) // 256 for n in sizes]
        c["m"] = [normal(gen, (n,), torch.float32, 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for n in sizes]
        c["v"] = [(torch.rand(n, generator=gen, device=DEV) * 448).to(torch.float8_e4m3fn).view(torch.uint8) for n in sizes]
        c["ms"], c["rs"] = ([torch.rand(b, generator=gen, device=DEV) * 1e-5 + 1e-7 for b in blocks] for _ in range(2))
    else:
        c["m"] = [normal(gen, (n,), torch.float32, 1e-3) for n in sizes]
        c["v"] = [torch.rand(n, generator=gen, device=DEV) * 1e-6 for n in sizes]
    c["table"] = N.adamw_tensors(c["p"], c["g"], c["m"], c["v"], c["master"], c["ms"], c["rs"])
    return c


def adam_want(c, i, lr, b1, b2, eps, wd, step, gs):
    """Values and bounds in 64 bits of tensor i before the step: p, m and v (or the root r)."""
    g = c["g"][i].double() * gs
    if c["ms"] is not None:
        m0, v0 = dequantise(c["m"][i], c["ms"][i]), dequantise(c["v"][i], c["rs"][i]).square()
    else:
        m0, v0 = c["m"][i].double(), c["v"][i].double()
    m, v = b1 * m0 + (1 - b1) * g, b2 * v0 + (1 - b2) * g * g
    w = (c["master"] or c["p"])[i].double()
    mag = (m0.abs() * b1 + (1 - b1) * g.abs())
    low = (v / (1 - b2 ** step)).sqrt() + eps
    move = lr / (1 - b1 ** step) * m / low
    # 16 A: under 16 fp32 roundings on the way to m, v and the update
    tmove = 16 * A * (lr / (1 - b1 ** step) * mag / low + move.abs())
    p = w - lr * wd * w - move
    return {"p": (p, tmove + 2 * A * (w.abs() + p.abs())), "m": (m, 16 * A * mag), "v": (v, 16 * A * v)}


ADAM = [
    ([1], "f32", "f32", False, "f32"), ([7, 256, 257, 8192, 8193], "f32", "bf16", False, "f32"),
    ([1, 8, 2047, 30_000], "bf16", "bf16", False, "f32"), ([300, 5], "bf16", "f32", True, "f32"),
    ([100_003, 1], "bf16", "bf16", True, "f32"),
    ([1], "f32", "f32", False, "e4m3"), ([255, 256, 257, 8192, 8193 + 256], "f32", "bf16", False, "e4m3"),
    ([3, 513, 40_001], "bf16", "bf16", False, "e4m3"), ([9, 2000], "bf16", "f32", False, "e4m3"),
    ([9, 2000], "bf16", "f32", True, "e4m3"), ([70_007], "bf16", "bf16", True, "e4m3"),
    ([5, 0, 70], "bf16", "f32", False, "f32"),
    (list(range(1, 100)), "bf16", "bf16", False, "f32"),  # more than one launch
]


@pytest.mark.parametrize("sizes,p,g,master,state", ADAM)
@pytest.mark.parametrize("device", [False, True])
def test_adamw(sizes, p, g, master, state, device):
    say("adamw", len(sizes), p, g, master, state, device)
    hyper = dict(lr=3e-3, b1=0.9, b2=0.95, eps=1e-8, wd=0.1, step=3)
    c = adam_case(sizes, p, g, master, state, seed=len(sizes))
    gs = torch.full((1,), 0.25, device=DEV) if device else None
    want = [adam_want(c, i, gs=0.25 if device else 1.0, **hyper) for i in range(len(sizes))]
    kw = dict(lr=hyper["lr"], step=hyper["step"])
    if device:
        kw = dict(lr=-1.0, step=0, lr_dev=torch.full((1,), hyper["lr"], device=DEV),
                  step_dev=torch.full((1,), hyper["step"], dtype=torch.int64, device=DEV), grad_scale=gs)
    N.moe_adamw(c["table"], beta1=hyper["b1"], beta2=hyper["b2"], eps=hyper["eps"], weight_decay=hyper["wd"], **kw)
    for i in range(len(sizes)):
        v, t = want[i]["p"]
        if master:
            check("master", c["master"][i], v, t)
        check("p", c["p"][i], v, t + half_step(DT[p]) * (v.abs() + t))
        if state == "f32":
            check("m", c["m"][i], *want[i]["m"])
            check("v", c["v"][i], *want[i]["v"])
            continue
        m, tm = want[i]["m"]
        r, tr = want[i]["v"][0].sqrt(), 16 * A * want[i]["v"][0].sqrt()
        for name, codes, scale, value, bound in (("m", c["m"][i], c["ms"][i], m, tm), ("r", c["v"][i], c["rs"][i], r, tr)):
            if not value.numel():
                continue
            block = torch.arange(value.numel(), device=DEV) // 256
            top = torch.zeros(scale.numel(), dtype=torch.float64, device=DEV).scatter_reduce_(0, block, value.abs(), "amax")
            far = torch.zeros_like(top).scatter_reduce_(0, block, bound, "amax")
            check(name + " scale", scale, top / 448, (far + 2 * A * top) / 448)
            # one step of e4m3: 2^-3 of the value, and 2^-9 of the scale under its normal range
            s = scale.double()[block]
            got = dequantise(codes, scale)
            check(name, got, value, bound + 4 * A * value.abs() + (value.abs() * 2.0 ** -3).clamp(min=s * 2.0 ** -9) * (1 + 8 * A))
            # the block's largest element keeps fp32 precision
            assert (codes.view(torch.float8_e4m3fn).float().abs().max() == 448)


def test_adamw_zero_state_and_zero_gradients():
    """The first step from zero states moves p by lr; dead elements (g = m = v = 0) stay, with eps and decay."""
    for state in ("f32", "e4m3"):
        n = 1000
        c = adam_case([n], "f32", "f32", False, state, seed=4)
        for name in ("m", "v"):
            c[name][0].zero_()
        if state == "e4m3":
            c["ms"][0].zero_()
            c["rs"][0].zero_()
        c["g"][0][500:] = 0
        before = c["p"][0].clone()
        N.moe_adamw(c["table"], lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-12, step=1)
        moved = (c["p"][0] - before)[:500]
        assert ((moved.abs() - 1e-2).abs() <= 1e-2 * 32 * A + 4 * A * before[:500].abs() + 1e-8).all()
        assert torch.equal(moved.sign(), -c["g"][0][:500].sign())
        assert torch.equal(c["p"][0][500:], before[500:])
        for _ in range(3):  # all-zero blocks keep finite scales and zero codes
            N.moe_adamw(c["table"], lr=1e-2, eps=1e-12, step=2)
        assert torch.equal(c["p"][0][768:], before[768:])


def test_adamw_tiny_gradients_without_eps():
    """v = 1e-41 is a denormal number of 7136 steps: the first update is lr within 2^-12 of it, in both formats."""
    for state in ("f32", "e4m3"):
        c = adam_case([700], "f32", "f32", False, state, seed=14)
        for name in ("m", "v", "ms", "rs"):
            if c[name] is not None:
                c[name][0].zero_()
        c["p"][0].zero_()
        c["g"][0].fill_(-1e-20)
        N.moe_adamw(c["table"], lr=1e-2, beta1=0.9, beta2=0.9, eps=0.0, step=1)
        # g^2 and v are rounded to 2^-149: 2^-17 and 2^-13.8 of them, half of that in the root
        assert ((c["p"][0] - 1e-2).abs() <= 1e-2 * 2.0 ** -12).all(), state


def test_adamw_non_finite_gradients_stay_in_their_elements():
    for state in ("f32", "e4m3"):
        c = adam_case([2000], "bf16", "bf16", False, state, seed=5)
        c["g"][0][3] = float("nan")
        c["g"][0][700] = float("inf")
        N.moe_adamw(c["table"], lr=1e-3, step=2)
        bad = ~torch.isfinite(c["p"][0].float())
        assert bad[3] and bad[700] and bad.sum() == 2
        c["g"][0].fill_(1e-3)  # nor do the states carry them to other elements of a block
        N.moe_adamw(c["table"], lr=1e-3, step=3)
        bad = ~torch.isfinite(c["p"][0].float())
        assert bad[3] and bad[700] and bad.sum() == 2


def test_adamw_captured_step_follows_device_values():
    """One captured call replayed: the step, the rate and the gradient scale come from device memory."""
    c, d = (adam_case([5000, 33], "bf16", "bf16", True, "e4m3", seed=6) for _ in range(2))
    lr, step = torch.full((1,), 1e-3, device=DEV), torch.ones(1, dtype=torch.int64, device=DEV)
    gs = torch.ones(1, device=DEV)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            N.moe_adamw(c["table"], weight_decay=0.1, lr_dev=lr, step_dev=step, grad_scale=gs)
    for t in range(1, 5):
        step.fill_(t)
        lr.fill_(1e-3 / t)
        gs.fill_(1.0 / t)
        graph.replay()
        torch.cuda.synchronize()
        N.moe_adamw(d["table"], weight_decay=0.1, lr_dev=lr, step_dev=step, grad_scale=gs)
        torch.cuda.synchronize()
        for name in ("p", "master", "m", "v", "ms", "rs"):
            assert all(torch.equal(x, y) for x, y in zip(c[name], d[name])), (t, name)


def test_adamw_8_bit_tracks_the_full_precision_run():
    """60 steps on gradients of fixed spread: the 8-bit run's update directions stay with the fp32 run's."""
    n, steps = 4096, 60
    gen = gen_of(7)
    spread = torch.exp(normal(gen, (n,), torch.float32))
    runs = {}
    for state in ("f32", "e4m3"):
        c = adam_case([n], "f32", "f32", False, state, seed=8)
        for name in ("m", "v", "ms", "rs"):
            if c[name] is not None:
                c[name][0].zero_()
        c["p"][0].zero_()
        g = gen_of(9)
        for t in range(1, steps + 1):
            c["g"][0].copy_(spread * (normal(g, (n,), torch.float32) + 0.5))
            N.moe_adamw(c["table"], lr=1e-3, beta2=0.95, step=t)
        runs[state] = c["p"][0].double()
    a, b = runs["f32"], runs["e4m3"]
    # A stored value is off by at most a step of 2^-3, at random, sqrt(1/6) of it in the mean square: 4% on
    # average steps of 0.09. The averages keep that as 4% / sqrt(1 - beta^2): 9% of m, 12% of r, correlated
    # over 1 / (1 - beta) = 10 and 20 of the 60 steps: 9% / sqrt(6) and 12% / sqrt(3) of the sum, 8% in all.
    assert (a - b).norm() <= 2.0 ** -3 * a.norm()


def words(n, seed, step):
    def f(z, s, t):
        w = (z ^ (z >> s)) * 0x85EBCA77 & 0xFFFFFFFF
        return w ^ (w >> t)
    key = f((seed + step * 0x9E3779B9) & 0xFFFFFFFF, 16, 13)
    return [f((i * 0x9E3779B1 + key) & 0xFFFFFFFF, 15, 13) for i in range(n)]


def test_adamw_random_rounding():
    """The stored codes are those of the stated rounding, and on average the value itself."""
    n = 4096
    c = adam_case([n], "f32", "f32", False, "e4m3", seed=10)
    for name in ("m", "v", "ms", "rs"):
        c[name][0].zero_()
    y = 448 * torch.exp2(-torch.rand(n, generator=gen_of(11), device=DEV) * 20)
    y[::256] = 448
    c["g"][0].copy_(y * torch.where(torch.arange(n, device=DEV) % 3 == 0, -1.0, 1.0))
    N.moe_adamw(c["table"], beta1=0.5, beta2=0.75, step=5, seed=0xFEDCBA98)  # m = g / 2, r = |g| / 2: exact
    x = torch.tensor(words(n, 0xFEDCBA98, 5), device=DEV)
    y = y.double()
    grid = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)
    for codes, bits, sign in ((c["m"][0], x >> 12, c["g"][0].double().sign()), (c["v"][0], x & 0xFFFFF, 1.0)):
        want = grid * torch.floor(y / grid + bits.double() / 2 ** 20) * sign
        got = codes.view(torch.float8_e4m3fn).double()
        # under 2^-6 the kernel rounds y + 2^-6 to fp32 first: 2^-30 of a grid of 2^-9, one value in 2^21
        assert (got != want).sum() <= 1
        # places are uniform: the mean error of n values is under 5 of its standard deviations, grid / sqrt(6 n)
        assert ((got - y * sign) / grid).mean().abs() <= 5 / (6 * n) ** 0.5


def test_adamw_slow_decay_reaches_the_codes():
    """With zero gradients r falls by sqrt(beta2) a step, also where that is less than half a code step."""
    n, steps = 8192, 40
    c = adam_case([n], "f32", "f32", False, "e4m3", seed=12)
    c["m"][0].zero_()
    c["v"][0].copy_((torch.rand(n, generator=gen_of(13), device=DEV) * 100 + 50).to(torch.float8_e4m3fn).view(torch.uint8))
    c["rs"][0].fill_(1e-5)
    hold = torch.arange(n, device=DEV) % 256 == 0  # one element per block keeps the block's scale
    c["v"][0][hold] = torch.full((1,), 448.0, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8)
    c["g"][0].zero_()
    c["g"][0][hold] = 448e-5
    start = dequantise(c["v"][0], c["rs"][0])
    for t in range(steps):
        N.moe_adamw(c["table"], beta1=0.9, beta2=0.98, step=t + 1, seed=3)
    end = dequantise(c["v"][0], c["rs"][0])
    ratio = (end / start)[~hold].mean().item()
    # per step a random error of at most 2^-3 of r, its square's mean 2^-3^2 / 6 < 0.003 wide; 40 of them over
    # 8160 elements leave the mean within 5 sqrt(40 * 0.003 / 8160) = 0.02, relative
    assert abs(ratio / 0.98 ** (steps / 2) - 1) <= 0.02


# ------------------------------------------------------------------------------------------------
# the layer

LAYERS = [
    L.LayerSpec("train-f32", T=24, H=256, E=6, k=2, I=128, act="f32", w_routed="f32", w_shared="f32", seed=61),
    L.LayerSpec("train-bf16-shared", T=100, H=512, E=8, k=3, I=256, shared=True, seed=62),
]


@pytest.mark.parametrize("spec", LAYERS, ids=[s.name for s in LAYERS])
@pytest.mark.parametrize("state,master", [("f32", False), ("e4m3", False), ("e4m3", True)])
def test_training_steps_of_a_layer(spec, state, master):
    """Forward, backward and AdamW together against 64-bit autograd of the same routing, two steps."""
    if master and spec.act == "f32":
        pytest.skip("fp32 weights take no master copy")
    say("layer", spec.name, state, master)
    gen, dtype = gen_of(spec.seed), DT[spec.act]
    H, I, E, k, T = spec.H, spec.I, spec.E, spec.k, spec.T

    def mats(*lead):
        return {"gate": normal(gen, (*lead, H, I), dtype, H ** -0.5), "up": normal(gen, (*lead, H, I), dtype, H ** -0.5),
                "down": normal(gen, (*lead, I, H), dtype, I ** -0.5)}
    routed, shared = mats(E), mats() if spec.shared else None
    lay = TrainableLayer(spec, normal(gen, (H, E), dtype, H ** -0.5), routed, shared, state=state, master=master)
    un = half_step(dtype)
    for step in range(2):
        x, dy = normal(gen, (T, H), dtype), normal(gen, (T, H), dtype)
        y = lay.forward(x)
        dx, dw = lay.backward(dy)
        idx = lay.idx.long()
        leaves = {"x": x.double().requires_grad_(), "w": lay.w.double().requires_grad_()}
        for tag, m in (("r", routed), ("s", shared)):
            if m is not None:
                leaves |= {tag + n: t.double().requires_grad_() for n, t in m.items()}
        rows = []
        for e in range(E):
            g = leaves["x"] @ leaves["rgate"][e]
            rows.append((g * torch.sigmoid(g) * (leaves["x"] @ leaves["rup"][e])) @ leaves["rdown"][e])
        picked = torch.stack(rows, 1).gather(1, idx[:, :, None].expand(T, k, H))
        want = (picked * leaves["w"][:, :, None]).sum(1)
        if shared is not None:
            g = leaves["x"] @ leaves["sgate"]
            want = want + (g * torch.sigmoid(g) * (leaves["x"] @ leaves["sup"])) @ leaves["sdown"]
        want.backward(dy.double())
        got = {"x": dx, "w": dw} | {"r" + n: t for n, t in lay.grads[0].items()}
        if shared is not None:
            got |= {"s" + n: t for n, t in lay.grads[1].items()}
        # up to 8 roundings of half a step on each path (g, u, h, y_perm, dy_perm, dg, du, the output), in norm
        tol = 8 * un + 1e-5

        def far(a, b):
            return ((a.double() - b).norm() / b.norm()).item()
        assert far(y, want.detach()) <= tol
        for n, t in got.items():
            assert far(t, leaves[n].grad) <= tol, n
        before = [t.double().clone() for t in lay.optimizer.keep[0]]
        lay.step(1e-2, weight_decay=0.0)
        for t, b, g in zip(lay.optimizer.keep[0], before, lay.optimizer.keep[1]):
            # |update| <= lr / (1 - b1^t) sqrt(sum of squares of the weights) <= 1.7 lr for these betas
            move = t.double() - b
            assert (move.abs() <= 1.7e-2 + un * (b.abs() + 2e-2)).all() and move.abs().max() > 5e-3
            if step == 0:
                big = g.double().abs() > 1e-6
                assert (move[big] * g.double()[big] <= 0).all()
    # another batch size on the same weights
    lay.set_tokens(T // 2 + 1)
    with pytest.raises(RuntimeError):
        lay.backward(dy)
    x = normal(gen, (T // 2 + 1, H), dtype)
    assert torch.isfinite(lay.forward(x).float()).all()


@pytest.mark.parametrize("spec", LAYERS, ids=[s.name for s in LAYERS])
def test_captured_training_step_of_a_layer(spec):
    """Routing, forward, backward and AdamW in one graph, replayed between eager steps of a second layer with the
    same weights: the same bits in every weight after every step."""
    say("captured layer", spec.name)
    dtype = DT[spec.act]
    H, I, E, T = spec.H, spec.I, spec.E, spec.T

    def build():
        gen = gen_of(spec.seed)

        def mats(*lead):
            return {"gate": normal(gen, (*lead, H, I), dtype, H ** -0.5), "up": normal(gen, (*lead, H, I), dtype, H ** -0.5),
                    "down": normal(gen, (*lead, I, H), dtype, I ** -0.5)}
        Wr = normal(gen, (H, E), dtype, H ** -0.5)
        return TrainableLayer(spec, Wr, mats(E), mats() if spec.shared else None, state="e4m3")
    a, b = build(), build()
    gen = gen_of(3)
    x, dy = normal(gen, (T, H), dtype), normal(gen, (T, H), dtype)
    step = torch.ones(1, dtype=torch.int64, device=DEV)

    def run(lay):
        y = lay.forward(x)
        dx, _ = lay.backward(dy)
        lay.step(1e-3, weight_decay=0.1, step_dev=step)
        return y, dx
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out = run(a)
    for t in range(1, 5):
        step.fill_(t)
        x.copy_(normal(gen, (T, H), dtype))
        graph.replay()
        torch.cuda.synchronize()
        want = run(b)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want)), t
        assert all(torch.equal(p, q) for p, q in zip(a.optimizer.keep[0], b.optimizer.keep[0])), t


def test_layer_on_another_stream_and_without_tokens():
    spec = LAYERS[1]
    gen, dtype = gen_of(1), DT[spec.act]
    H, I, E = spec.H, spec.I, spec.E
    routed = {"gate": normal(gen, (E, H, I), dtype, H ** -0.5), "up": normal(gen, (E, H, I), dtype, H ** -0.5),
              "down": normal(gen, (E, I, H), dtype, I ** -0.5)}
    with pytest.raises(ValueError):
        TrainableLayer(spec, normal(gen, (H, E), dtype), routed | {"up": routed["down"]})
    lay = TrainableLayer(spec, normal(gen, (H, E), dtype, H ** -0.5), routed)
    x, dy = normal(gen, (spec.T, H), dtype), normal(gen, (spec.T, H), dtype)
    with pytest.raises(ValueError):
        lay.forward(x[:-1])
    want = lay.forward(x), *lay.backward(dy)
    want = [t.clone() for t in want]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lay.forward(x, stream=side), *lay.backward(dy, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    lay.set_tokens(0)
    assert lay.forward(x[:0]).shape == (0, H)
    dx, dw = lay.backward(dy[:0])
    assert dx.shape == (0, H) and all((t == 0).all() for t in lay.grads[0].values())
