"""What include/moe.h and TrainableLayer promise about training beside the formulas, on the GPU."""
import pytest
import torch

from expert_ffn_layer_amd import native as N
from expert_ffn_layer_amd.layer import TrainableLayer
from inputgen import layers as L

from _gpu import say
from _train import DT, backward, chain_error, check

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def gen_of(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)


# ------------------------------------------------------------------------------------------------
# AdamW

def is_nan_code(codes):
    return (codes & 0x7F) == 0x7F


@pytest.mark.parametrize("g,word", [("bf16", 0x7FFF), ("bf16", 0xFFFF), ("bf16", 0x7FC0), ("bf16", 0x7F80), ("bf16", 0xFF80),
                                    ("f32", 0x7FFFFFFF), ("f32", 0xFFFFFFFF), ("f32", 0x7FC00001), ("f32", 0x7F800000)])
def test_adamw_8_bit_states_keep_every_nan(g, word):
    """m and sqrt(v) become NaN exactly where the gradient is NaN or infinite, whatever the NaN's payload, and stay so."""
    say("nan codes", g, hex(word))
    n = 20_000
    gen = gen_of(word)
    p, grad = normal(gen, (n,), torch.bfloat16, 0.05), normal(gen, (n,), DT[g], 1e-3)
    at = torch.rand(n, generator=gen, device=DEV) < 0.1
    bits = grad.view(torch.int16 if g == "bf16" else torch.int32)
    bits[at] = word - (1 << 16) if g == "bf16" and word >> 15 else word - (1 << 32) if word >> 31 else word
    m, v = (torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2))
    ms, vs = (torch.zeros((n + 255) // 256, device=DEV) for _ in range(2))
    table = N.adamw_tensors([p], [grad], [m], [v], None, [ms], [vs])
    for step in range(1, 9):
        N.moe_adamw(table, lr=1e-3, step=step, seed=1000 * step)
        if step == 4:
            grad.fill_(1e-3)
        assert torch.equal(is_nan_code(m), at) and torch.equal(is_nan_code(v), at), step
        assert torch.equal(torch.isnan(p), at), step
        assert torch.isfinite(ms).all() and torch.isfinite(vs).all()


@pytest.mark.parametrize("state", ["f32", "e4m3"])
@pytest.mark.parametrize("eps", [1e-44, 1e-39, 2.0 ** -126])
def test_adamw_smallest_eps(state, eps):
    """Elements without gradient stay where they are by any eps that is accepted (0 / eps = 0); one that a reciprocal
    in fp32 cannot take is refused."""
    say("eps", state, eps)
    n = 300
    p, g = torch.ones(n, device=DEV), torch.zeros(n, device=DEV)
    q8 = state == "e4m3"
    m, v = (torch.zeros(n, dtype=torch.uint8 if q8 else torch.float32, device=DEV) for _ in range(2))
    scales = [[torch.zeros(2, device=DEV)] for _ in range(2)] if q8 else [None, None]
    table = N.adamw_tensors([p], [g], [m], [v], None, *scales)
    if eps < 2.0 ** -126:
        with pytest.raises(N.MoeError):
            N.moe_adamw(table, lr=1e-3, eps=eps, step=1)
    else:
        N.moe_adamw(table, lr=1e-3, eps=eps, step=1)
    assert (p == 1).all()


@pytest.mark.parametrize("q8", [False, True])
def test_adamw_takes_arrays_side_by_side(q8):
    """All arrays of two tensors packed without a gap, and one gradient for both: the same bits as apart."""
    say("packed arrays", q8)
    n, size = 512, torch.uint8 if q8 else torch.float32

    def run(packed):
        block = torch.zeros(64 * 1024, dtype=torch.uint8, device=DEV)
        at = [0]

        def take(count, dtype):
            b = count * torch.empty(0, dtype=dtype).element_size()
            if not packed:
                return torch.zeros(count, dtype=dtype, device=DEV)
            t = block[at[0]:at[0] + b].view(dtype)
            at[0] += b
            return t
        p, m, v = [take(n, torch.bfloat16) for _ in range(2)], [take(n, size) for _ in range(2)], [take(n, size) for _ in range(2)]
        ms, vs = ([take(n // 256, torch.float32) for _ in range(2)] for _ in range(2)) if q8 else (None, None)
        g = take(n, torch.bfloat16)
        g.copy_(normal(gen_of(4), (n,), torch.bfloat16))
        for i in range(2):
            p[i].copy_(normal(gen_of(i), (n,), torch.bfloat16))
        N.moe_adamw(N.adamw_tensors(p, [g, g], m, v, None, ms, vs), lr=1e-2, step=1)
        return [t.clone() for t in (*p, *m, *v, *(ms or []), *(vs or []))]
    assert all(torch.equal(a, b) for a, b in zip(run(True), run(False)))


# ------------------------------------------------------------------------------------------------
# the layer

SPEC = L.LayerSpec("train-contract", T=100, H=512, E=8, k=3, I=256, shared=True, seed=62)


def build_layer(spec=SPEC, seed=1, **kw):
    gen, dtype = gen_of(seed), DT[spec.act]
    H, I, E = spec.H, spec.I, spec.E

    def mats(*lead):
        return {"gate": normal(gen, (*lead, H, I), dtype, H ** -0.5), "up": normal(gen, (*lead, H, I), dtype, H ** -0.5),
                "down": normal(gen, (*lead, I, H), dtype, I ** -0.5)}
    Wr = normal(gen, (H, E), dtype, H ** -0.5)
    return TrainableLayer(spec, Wr, mats(E), mats() if spec.shared else None, **kw)


def batch(spec, seed, T=None):
    gen = gen_of(seed)
    return [normal(gen, (spec.T if T is None else T, spec.H), DT[spec.act]) for _ in range(2)]


def test_layer_results_outlive_the_next_batch():
    say("results")
    lay = build_layer()
    kept, copies = [], []
    for seed in range(3):
        x, dy = batch(SPEC, seed)
        y = lay.forward(x)
        out = (y, *lay.backward(dy))
        kept.append(out)
        copies.append([t.clone() for t in out])
    for out, want in zip(kept, copies):
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_layer_counts_the_steps_it_made():
    """A refused step is none: the next one is the first."""
    say("refused step")
    a, b = build_layer(), build_layer()
    for lay in (a, b):
        x, dy = batch(SPEC, 3)
        lay.forward(x)
        lay.backward(dy)
    with pytest.raises(N.MoeError):
        a.step(-1.0)
    with pytest.raises(ValueError):
        a.step(1e-3, step_dev=torch.ones(1, device=DEV))
    a.step(1e-3)
    b.step(1e-3)
    assert a.steps == 1 and all(torch.equal(p, q) for p, q in zip(a.optimizer.keep[0], b.optimizer.keep[0]))


def test_layer_step_refuses_device_values_on_the_host():
    say("host values")
    lay = build_layer()
    for kw in (dict(lr_dev=torch.ones(1)), dict(step_dev=torch.ones(1, dtype=torch.int64)), dict(grad_scale=torch.ones(1))):
        with pytest.raises(ValueError):
            lay.step(1e-3, **kw)
    assert lay.steps == 0


def busy(stream):
    """Some 20 ms of other work on the stream, so that what follows waits behind it."""
    a = torch.ones((8192, 8192), dtype=torch.bfloat16, device=DEV)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(20):
            b = a @ a
    return a, b


def overwrite(like):
    """New tensors of the current stream in the place of freed ones of the same sizes."""
    return [torch.full(shape, 3.0, dtype=dtype, device=DEV) for shape, dtype in like for _ in range(3)]


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("what", ["set_tokens", "next batch", "layer"])
def test_memory_stays_until_its_stream_is_through(what, given):
    """What a call on a side stream still has to read is dropped, and memory of those sizes written, without a host
    synchronisation; given: the stream as an argument, otherwise as the current one."""
    say("memory", what, given)
    want_layer, lay = build_layer(), build_layer()
    x, dy = batch(SPEC, 5)
    want = [want_layer.forward(x), *want_layer.backward(dy)]
    want_layer.step(1e-3)
    want += [t.clone() for t in want_layer.optimizer.keep[0]]
    sizes = [(t.shape, t.dtype) for t in (x, lay.ws, lay.idx, lay.w, lay.off, lay.slot_token, lay.dy_perm, *lay.y, *lay.dx,
                                         *lay.pre[0], *lay.optimizer.keep[1], *lay.optimizer.keep[2])]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    kept = busy(side)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(None if given else side):
        kw = dict(stream=side) if given else {}
        got = [lay.forward(x, **kw), *lay.backward(dy, **kw)]
        lay.step(1e-3, **kw)
        got += lay.optimizer.keep[0]
        if what == "next batch":
            lay.forward(dy, **kw)
    del x, dy
    if what == "set_tokens":
        lay.set_tokens(SPEC.T)
    elif what == "layer":
        del lay
    new = overwrite(sizes)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all((t == 3).all() for t in new)
    del kept


def test_set_tokens_on_a_stream():
    """Buffers made and filled on the stream that uses them, behind other work there."""
    say("set_tokens on a stream")
    want_layer, lay = build_layer(), build_layer()
    T = 57
    x, dy = batch(SPEC, 7, T)
    want_layer.set_tokens(T)
    want = [want_layer.forward(x), *want_layer.backward(dy)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    kept = busy(side)
    lay.set_tokens(T, stream=side)
    got = [lay.forward(x, stream=side), *lay.backward(dy, stream=side)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del kept


# ------------------------------------------------------------------------------------------------
# the error of the fp32 products. Gates of 32 and more make the sigmoid 1 in fp32, so that what goes into a product is
# known to a rounding.

def far(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


def f32_block(T, H, I, seed):
    gen = gen_of(seed)
    shape = N.make_shape(T, H, 1, 1, I, act="f32", w_routed="f32")
    w = {"gate": normal(gen, (1, H, I), torch.float32), "up": normal(gen, (1, H, I), torch.float32),
         "down": normal(gen, (1, I, H), torch.float32)}
    return gen, shape, w, torch.empty(N.moe_train_workspace_size(shape), dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("H,T", [(640, 100), (7168, 100), (7168, 2000)])
def test_f32_error_of_gate_and_up(H, T):
    say("f32 gate/up", H, T)
    gen, shape, w, ws = f32_block(T, H, 128, 31)
    x = normal(gen, (T, H), torch.float32)
    g, u, y = (torch.empty((T, n), device=DEV) for n in (128, 128, H))
    N.moe_gated_ffn(shape, x, None, None, w, g, u, y, ws)
    for got, name in ((g, "gate"), (u, "up")):
        error = far(got, x.double() @ w[name][0].double())
        say(name, error / 2.0 ** -24)
        assert error <= chain_error(H)


@pytest.mark.parametrize("I,T", [(640, 128), (8192, 128), (8192, 2048)])
def test_f32_error_of_down(I, T):
    """Each row of x picks a row of the weights, so g and u are exact and h has one rounding."""
    say("f32 down", I, T)
    H = 128
    gen, shape, w, ws = f32_block(T, H, I, 32)
    w["gate"] = torch.rand((1, H, I), generator=gen, device=DEV) * 32 + 32
    pick = torch.arange(T, device=DEV) % H
    x = torch.eye(H, device=DEV)[pick].contiguous()
    y = torch.empty((T, H), device=DEV)
    N.moe_gated_ffn(shape, x, None, None, w, None, None, y, ws)
    h = (w["gate"][0].double() * w["up"][0].double())[pick]
    error = far(y, h @ w["down"][0].double())
    say(error / 2.0 ** -24)
    assert error <= chain_error(I)


@pytest.mark.parametrize("I,T", [(384, 128), (4096, 128), (4096, 2048)])
def test_f32_error_of_dx(I, T):
    """Each row of dy picks a column of Wd, so dh is exact, du = 64 dh too, and dg = dh u has one rounding."""
    say("f32 dx", I, T)
    H = 128
    gen, shape, w, ws = f32_block(T, H, I, 33)
    pick = torch.arange(T, device=DEV) % H
    dy = torch.eye(H, device=DEV)[pick].contiguous()
    g, u = torch.full((T, I), 64.0, device=DEV), normal(gen, (T, I), torch.float32, 64.0)
    x, dx = normal(gen, (T, H), torch.float32), torch.empty((T, H), device=DEV)
    N.moe_gated_ffn_backward(shape, x, None, None, w, g, u, dy, dx, None, ws)
    dh = w["down"][0].double().T[pick]
    want = (dh * u.double()) @ w["gate"][0].double().T + (dh * 64) @ w["up"][0].double().T
    error = far(dx, want)
    say(error / 2.0 ** -24)
    assert error <= chain_error(2 * I)


@pytest.mark.parametrize("T", [1000, 20_000, 140_000])
def test_f32_error_of_the_weight_gradients(T):
    """h = 64 u is exact, du = 64 dh and dg = dh u are as far off as dh."""
    say("f32 weight gradients", T)
    H = I = 128
    gen, shape, w, ws = f32_block(T, H, I, 34)
    x, dy = normal(gen, (T, H), torch.float32), normal(gen, (T, H), torch.float32)
    g, u = torch.full((T, I), 64.0, device=DEV), normal(gen, (T, I), torch.float32)
    grads = {n: torch.empty_like(t) for n, t in w.items()}
    N.moe_gated_ffn_backward(shape, x, None, None, w, g, u, dy, None, grads, ws)
    dh = dy.double() @ w["down"][0].double().T
    want = {"gate": x.double().T @ (dh * u.double()), "up": x.double().T @ (dh * 64), "down": (64 * u.double()).T @ dy.double()}
    for name, bound in (("gate", chain_error(H, T)), ("up", chain_error(H, T)), ("down", chain_error(T))):
        error = far(grads[name][0], want[name])
        say(name, error / 2.0 ** -24)
        assert error <= bound, name


# ------------------------------------------------------------------------------------------------
# the binding

def test_binding_refuses_strided_tensors():
    """The library takes addresses, so a view of other strides would be read as another matrix."""
    say("strides")
    T, H, I = 8, 256, 128
    shape = N.make_shape(T, H, 1, 1, I)
    gen = gen_of(5)
    b = {"x": normal(gen, (T, H), torch.bfloat16), "g": normal(gen, (T, I), torch.bfloat16), "u": normal(gen, (T, I), torch.bfloat16),
         "dy": normal(gen, (T, H), torch.bfloat16), "y": torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)}
    w = {"gate": normal(gen, (1, H, I), torch.bfloat16), "up": normal(gen, (1, H, I), torch.bfloat16),
         "down": normal(gen, (1, I, H), torch.bfloat16)}
    grads = {n: torch.zeros_like(t) for n, t in w.items()}
    ws = torch.empty(N.moe_train_workspace_size(shape), dtype=torch.uint8, device=DEV)

    def turned(t):  # the same values under other strides
        return t.transpose(-1, -2).contiguous().transpose(-1, -2)

    def forward(b, w):
        N.moe_gated_ffn(shape, b["x"], None, None, w, b["g"], b["u"], b["y"], ws)

    def backward(b, w, grads=grads):
        N.moe_gated_ffn_backward(shape, b["x"], None, None, w, b["g"], b["u"], b["dy"], b["y"], grads, ws)
    forward(b, w)
    backward(b, w)
    for call, names in ((forward, "xguy"), (backward, ("x", "g", "u", "dy", "y"))):
        for n in names:
            with pytest.raises(ValueError):
                call(b | {n: turned(b[n])}, w)
        for n in w:
            with pytest.raises(ValueError):
                call(b, w | {n: turned(w[n])})
    for n in w:
        with pytest.raises(ValueError):
            backward(b, w, grads | {n: turned(grads[n])})
    slot, one = torch.zeros((T, 1), dtype=torch.int32, device=DEV), torch.ones((T, 1), device=DEV)
    rows = torch.zeros_like(b["y"])
    N.moe_combine_backward(shape, b["dy"], b["y"], slot, one, rows, torch.zeros_like(one))
    with pytest.raises(ValueError):
        N.moe_combine_backward(shape, turned(b["dy"]), b["y"], slot, one, rows, torch.zeros_like(one))


# ------------------------------------------------------------------------------------------------
# arguments side by side

@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_block_takes_arguments_side_by_side(act):
    """Every argument of the block and its gradient packed without a gap: the same bits as apart; and the combine's
    gradient with the routing weights' in their place."""
    say("packed block", act)
    T, H, I, E, k = 24, 256, 128, 3, 2
    P, dtype = T * k, DT[act]
    shape = N.make_shape(T, H, E, k, I, act=act, w_routed=act)
    size = N.moe_train_workspace_size(shape)

    def run(packed):
        gen, at = gen_of(8), [0]
        memory = torch.zeros(8 << 20, dtype=torch.uint8, device=DEV)

        def take(*dims, dtype=dtype):
            n = torch.Size(dims).numel()
            b = n * torch.empty(0, dtype=dtype).element_size()
            if not packed:
                return torch.zeros(dims, dtype=dtype, device=DEV)
            t = memory[at[0]:at[0] + b].view(dtype).view(dims)
            at[0] += b
            return t

        def filled(*dims):
            return take(*dims).copy_(normal(gen, dims, dtype))
        ws = take(size, dtype=torch.uint8)
        x, g, u, y = filled(T, H), take(P, I), take(P, I), take(P, H)
        w = {"gate": filled(E, H, I), "up": filled(E, H, I), "down": filled(E, I, H)}
        grads = {n: take(*t.shape) for n, t in w.items()}
        dy, dx, rows = filled(T, H), take(P, H), take(P, H)
        tw, dw = take(T, k, dtype=torch.float32), take(T, k, dtype=torch.float32)
        tw.copy_(torch.rand((T, k), generator=gen, device=DEV))
        slot, pair = take(P, dtype=torch.int32), take(P, dtype=torch.int32)
        slot.copy_(torch.arange(P, device=DEV, dtype=torch.int32) % T)
        pair.copy_(torch.randperm(P, generator=gen, device=DEV))
        off = take(E + 1, dtype=torch.int32)
        off.copy_(torch.tensor([0, 20, 20, P]))
        N.moe_gated_ffn(shape, x, off, slot, w, g, u, y, ws)
        if packed:
            N.moe_combine_backward(shape, dy, y, pair, tw, rows, tw)
        else:
            N.moe_combine_backward(shape, dy, y, pair, tw, rows, dw)
        N.moe_gated_ffn_backward(shape, x, off, slot, w, g, u, rows, dx, grads, ws)
        return [t.clone() for t in (g, u, y, rows, tw if packed else dw, dx, *grads.values())]
    assert all(torch.equal(a, b) for a, b in zip(run(True), run(False)))


# ------------------------------------------------------------------------------------------------
# large calls

@pytest.mark.slow
def test_gradient_of_the_most_rows():
    """The most rows that a call takes, of a width that puts P H / 8, the threads of the gathering of x, past 2^32: the
    gradients of the last rows, which a group of their own holds, against their definition."""
    T, k, E, H, I, last = 262140, 16, 16, 8320, 128, 75
    P = T * k
    assert P == 65535 * 64 and P * H // 8 > 1 << 32
    torch.cuda.empty_cache()
    shape = N.make_shape(T, H, E, k, I)
    size = N.moe_train_workspace_size(shape)
    if torch.cuda.mem_get_info()[0] < size + P * H * 2 + (20 << 30):
        pytest.skip("needs 150 GB of GPU memory")
    say("most rows", P, H)
    gen = gen_of(3)
    x = normal(gen, (T, H), torch.bfloat16)
    w = {"gate": normal(gen, (E, H, I), torch.bfloat16, H ** -0.5), "up": normal(gen, (E, H, I), torch.bfloat16, H ** -0.5),
         "down": normal(gen, (E, I, H), torch.bfloat16, I ** -0.5)}
    g, u = (torch.zeros((P, I), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    dy = torch.zeros((P, H), dtype=torch.bfloat16, device=DEV)
    for t, n in ((g, I), (u, I), (dy, H)):
        t[P - last:] = normal(gen, (last, n), torch.bfloat16)
    slot = torch.arange(P, dtype=torch.int32, device=DEV) % T
    off = torch.full((E + 1,), P - last, dtype=torch.int32, device=DEV)
    off[0], off[E] = 0, P
    grads = {n: torch.full_like(t, 5.0) for n, t in w.items()}
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    N.moe_gated_ffn_backward(shape, x, off, slot, w, g, u, dy, None, grads, ws)
    torch.cuda.synchronize()
    assert all((t[:E - 1] == 0).all() for t in grads.values())
    rows = x[slot[P - last:].long()].double()
    mats = [w[n][E - 1].double() for n in ("gate", "up", "down")]
    want = backward(rows, *mats, g[P - last:].double(), u[P - last:].double(), dy[P - last:].double(), torch.bfloat16)
    for n in ("gate", "up", "down"):
        check("d" + n, grads[n][E - 1], *want["d" + n])
    del ws, dy, g, u, x
    torch.cuda.empty_cache()
