"""What training one MoE expert-FFN layer needs beside its forward pass: the gated feed-forward block that
keeps what its gradient reads, that gradient, the gradient of the weighted combine, and the AdamW step.

``own`` chooses between the framework's entry points and the same operators in elementary torch operations."""
import math

import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BLOCK = 256  # elements of an optimizer state that share a scale in the 8-bit form


# ------------------------------------------------------------------------------------------------
# cases

def ffn(name, op, T, H, I, E, k, act="bf16", skew=0.0, skip=0.0):
    c = {"op": op, "T": T, "H": H, "I": I, "E": E, "k": k, "act": act, "skew": skew, "skip": skip}
    return {"name": name, **c} if name else c


def comb(name, T, H, k, act="bf16", skip=0.0):
    c = {"op": "combine_backward", "T": T, "H": H, "k": k, "act": act, "skip": skip}
    return {"name": name, **c} if name else c


def adam(name, sizes, p="bf16", g="bf16", master=False, state="f32", scaled=False):
    c = {"op": "adamw", "sizes": sizes, "p": p, "g": g, "master": master, "state": state, "scaled": scaled}
    return {"name": name, **c} if name else c


def listed():
    return [
        # the tiny fp32 layer: what a user's gradient check runs; launch latency counts
        ffn("ffn tiny f32", "ffn", 16, 256, 128, 8, 2, "f32"),
        # few rows per expert on a Qwen3-shaped slice of 16 experts: bound by reading the weights
        ffn("ffn thin groups", "ffn", 61, 4096, 1536, 16, 8, skew=0.5, skip=0.1),
        # one dense block (a shared expert) on an odd number of tokens
        ffn("ffn dense", "ffn", 1027, 4096, 1536, 1, 1),
        # a 32-expert slice of the DeepSeek-V3 layer: the bulk of a training step's forward
        ffn("ffn grouped", "ffn", 4096, 7168, 2048, 32, 8, skew=0.3),
        # the gradient of a small fp32 layer with odd groups
        ffn("ffn backward f32", "ffn_backward", 333, 1024, 384, 5, 2, "f32", skew=1.0),
        # the gradient of the dense block
        ffn("ffn backward dense", "ffn_backward", 1027, 4096, 1536, 1, 1),
        # the gradient of the V3 slice: the bulk of a training step
        ffn("ffn backward grouped", "ffn_backward", 4096, 7168, 2048, 32, 8, skew=0.3),
        # combine of a small batch, some pairs held by other GPUs
        comb("combine backward small", 64, 4096, 8, skip=0.1),
        # combine of the 16384-token V3 batch
        comb("combine backward large", 16384, 7168, 8),
        # the tiny layer's tensors: three expert matrices, the router and its bias, all fp32
        adam("adamw tiny", "262144x3,2048,8", "f32", "f32"),
        # twelve V3 expert matrices, a router and two vectors in bf16 with fp32 master weights; clipped gradients
        adam("adamw master", "14680064x12,1835008,7168,257", master=True, scaled=True),
        # the same matrices with 8-bit states
        adam("adamw 8-bit", "14680064x10,1835008,257", state="q8"),
    ]


def spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn_backward", "ffn_backward", "combine_backward", "adamw", "adamw"])
    if op in ("ffn", "ffn_backward"):
        act = rng.choice(["bf16", "bf16", "bf16", "f32"])
        E = rng.choice([1, spread(rng, 2, 48)])
        k = 1 if E == 1 else rng.randint(1, min(8, E))
        H = 128 * spread(rng, 2, 56 if act == "bf16" else 16)
        I = 128 * spread(rng, 1, 16 if act == "bf16" else 8)
        while E * H * I > 32 * 7168 * 2048:
            E = max(1, E // 2)
            k = min(k, E)
        T = spread(rng, 1, 4096)
        while T * k > (32768 if act == "bf16" else 4096):
            T = max(1, T // 2)
        return ffn(None, op, T, H, I, E, k, act, skew=round(rng.uniform(0.0, 1.0), 2) if T * k < 4096 else 0.3,
                   skip=rng.choice([0.0, 0.0, 0.2]) if E > 1 else 0.0)
    if op == "combine_backward":
        T, H = spread(rng, 1, 16384), 128 * spread(rng, 2, 56)
        return comb(None, T, H, rng.randint(1, 8), rng.choice(["bf16", "bf16", "f32"]) if T <= 4096 else "bf16",
                    skip=rng.choice([0.0, 0.2]))
    state = rng.choice(["f32", "q8"])
    sizes = ",".join(str(spread(rng, 1, 9_000_000)) for _ in range(rng.randint(1, 10)))
    p = rng.choice(["bf16", "bf16", "f32"])
    master = p == "bf16" and rng.random() < 0.4
    return adam(None, sizes, p, "f32" if p == "f32" else rng.choice(["bf16", "f32"]), master, state, rng.random() < 0.5)


def tensor_sizes(text):
    out = []
    for part in text.split(","):
        n, _, times = part.partition("x")
        out += [int(n)] * int(times or 1)
    return out


# ------------------------------------------------------------------------------------------------
# inputs

def routing(c, gen):
    """k distinct experts a token, popularity falling with the expert's index by `skew`, a share `skip` of the
    pairs held elsewhere; the rows of each expert in token order, as moe_permute lays them out."""
    T, E, k = c["T"], c["E"], c["k"]
    pop = -c["skew"] * torch.log1p(torch.arange(E, device=DEV, dtype=torch.float32))
    noise = -torch.log(-torch.log(torch.rand(T, E, device=DEV, generator=gen).clamp_(1e-9, 1 - 1e-7)))
    idx = (noise + pop).topk(k, dim=1).indices.sort(dim=1).values.reshape(-1)
    idx = torch.where(torch.rand(T * k, device=DEV, generator=gen) < c["skip"], E, idx)
    order = torch.sort(idx, stable=True).indices
    counts = torch.bincount(idx, minlength=E + 1)[:E]
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[1:] = counts.cumsum(0)
    n = int(off[E])
    slot_token = torch.zeros(T * k, dtype=torch.int32, device=DEV)
    slot_token[:n] = (order[:n] // k).int()
    return off, slot_token, n, max(1, int(counts.max()))


def normal(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, device=DEV, generator=gen) * std).to(dtype)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if c["op"] == "adamw":
        return prepare_adam(c, gen)
    dt = DT[c["act"]]
    T, H, k = c["T"], c["H"], c["k"]
    s = {"case": c}
    if c["op"] == "combine_backward":
        P = T * k
        slot = torch.randperm(P, device=DEV, generator=gen).int()
        gone = torch.rand(P, device=DEV, generator=gen) < c["skip"]
        s["n"] = int((~gone).sum())
        rank = torch.zeros(P, dtype=torch.int32, device=DEV)
        order = torch.where(gone, P, slot).sort().indices
        rank[order] = torch.arange(P, dtype=torch.int32, device=DEV)
        s["pair_slot"] = torch.where(gone, -1, rank).int().reshape(T, k).contiguous()
        w = torch.rand(T, k, device=DEV, generator=gen) + 0.05
        s["w"] = w / w.sum(1, keepdim=True)
        s["dy"], s["y_perm"] = normal(gen, (T, H), dt), normal(gen, (P, H), dt)
        s["dy_perm"] = torch.zeros(P, H, dtype=dt, device=DEV)
        s["dw"] = torch.zeros(T, k, dtype=torch.float32, device=DEV)
        return s
    E, I, P = c["E"], c["I"], T * k
    s["off"], s["slot"], s["n"], s["most"] = routing(c, gen)
    s["x"] = normal(gen, (T, H), dt)
    s["gate"], s["up"] = (normal(gen, (E, H, I), dt, H ** -0.5) for _ in range(2))
    s["down"] = normal(gen, (E, I, H), dt, I ** -0.5)
    if c["op"] == "ffn":
        s["g"], s["u"] = (torch.zeros(P, I, dtype=dt, device=DEV) for _ in range(2))
        s["y"] = torch.zeros(P, H, dtype=dt, device=DEV)
        return s
    s["g"], s["u"], s["dy"] = normal(gen, (P, I), dt), normal(gen, (P, I), dt), normal(gen, (P, H), dt, 0.1)
    s["dx"] = torch.zeros(P, H, dtype=dt, device=DEV)
    s["dgate"], s["dup"], s["ddown"] = (torch.zeros_like(s[n]) for n in ("gate", "up", "down"))
    return s


def prepare_adam(c, gen):
    s = {"case": c, "lr": 1e-4, "b1": 0.9, "b2": 0.95, "eps": 1e-8, "wd": 0.1, "step": 12}
    sizes = tensor_sizes(c["sizes"])
    w = [torch.randn(n, device=DEV, generator=gen) * 0.02 for n in sizes]
    s["p"] = [t.to(DT[c["p"]]) for t in w]
    s["master"] = w if c["master"] else []
    s["g"] = [normal(gen, (n,), DT[c["g"]], 1e-3) for n in sizes]
    s["scale"] = torch.full((1,), 0.37, device=DEV) if c["scaled"] else None
    m = [torch.randn(n, device=DEV, generator=gen) * 3e-4 for n in sizes]
    r = [torch.rand(n, device=DEV, generator=gen) * 1e-3 + 1e-5 for n in sizes]
    if c["state"] == "f32":
        s["m"], s["v"] = m, [t * t for t in r]
        return s
    s["seed"] = 77
    bits = [dither(n, 1, 1) for n in sizes]
    s["m"], s["ms"] = map(list, zip(*[quantised(t, x >> 12) for t, x in zip(m, bits)]))
    s["r"], s["rs"] = map(list, zip(*[quantised(t, x & 0xFFFFF) for t, x in zip(r, bits)]))
    return s


# ------------------------------------------------------------------------------------------------
# plain forms

def blocks(t):
    return torch.nn.functional.pad(t, (0, -t.numel() % BLOCK)).reshape(-1, BLOCK)


def dither(n, seed, step):
    """32 bits per element from its index, the seed and the step; m takes the upper 20, the root the lower 20."""
    key = (seed + step * 0x9E3779B9) & 0xFFFFFFFF
    key = (key ^ key >> 16) * 0x85EBCA77 & 0xFFFFFFFF
    x = (torch.arange(n, device=DEV) * 0x9E3779B1 + (key ^ key >> 13)) & 0xFFFFFFFF
    x = (x ^ x >> 15) * 0x85EBCA77 & 0xFFFFFFFF
    return x ^ x >> 13


def quantised(t, bits):
    """e4m3 codes of t over one float scale (the largest magnitude, at least 2^-100, / 448) per BLOCK elements:
    a value between two codes takes the upper one with a probability of its place between them, by 20 bits."""
    b = blocks(t)
    top = b.abs().amax(1).clamp(min=2.0 ** -100)
    y = (b * (448.0 / top)[:, None]).reshape(-1)[:t.numel()]
    low = torch.where(y.abs() < 2.0 ** -6, 2.0 ** -6, 0.0)  # there the codes are 2^-9 apart, as above 2^-6
    z = ((y.abs().clamp(max=448.0) + low).view(torch.int32) + bits.int()) & -0x100000
    return torch.copysign(z.view(torch.float32) - low, y).to(torch.float8_e4m3fn), top * (1.0 / 448.0)


def dequantised(codes, scale):
    return (blocks(codes.float()) * scale[:, None]).reshape(-1)[:codes.numel()]


def padded(rows, place, E, most):
    """The first rows of a [P][...] tensor, those of each group at the front of its own [most] rows, in fp32."""
    out = torch.zeros(E * most, rows.shape[1], dtype=torch.float32, device=rows.device)
    out[place] = rows.float()
    return out.reshape(E, most, -1)


def places(s):
    E, n = s["case"]["E"], s["n"]
    off = s["off"].long()
    group = torch.repeat_interleave(torch.arange(E, device=off.device), off[1:] - off[:-1], output_size=n)
    return group * s["most"] + torch.arange(n, device=off.device) - off[group]


def plain_ffn(s):
    c, n = s["case"], s["n"]
    place = places(s)
    x = padded(s["x"][s["slot"][:n].long()], place, c["E"], s["most"])
    g, u = x @ s["gate"].float(), x @ s["up"].float()
    y = (g / (1.0 + torch.exp(-g)) * u) @ s["down"].float()
    s["g"][:n] = g.reshape(-1, c["I"])[place].to(s["g"].dtype)
    s["u"][:n] = u.reshape(-1, c["I"])[place].to(s["u"].dtype)
    s["y"][:n] = y.reshape(-1, c["H"])[place].to(s["y"].dtype)
    return {"y": s["y"], "g": s["g"], "u": s["u"]}


def plain_ffn_backward(s):
    c, n = s["case"], s["n"]
    place = places(s)
    x = padded(s["x"][s["slot"][:n].long()], place, c["E"], s["most"])
    g, u, dy = (padded(s[name][:n], place, c["E"], s["most"]) for name in ("g", "u", "dy"))
    sig = 1.0 / (1.0 + torch.exp(-g))
    dh = dy @ s["down"].float().transpose(1, 2)
    du = dh * (g * sig)
    dg = dh * u * (sig * (1.0 + g * (1.0 - sig)))
    dx = dg @ s["gate"].float().transpose(1, 2) + du @ s["up"].float().transpose(1, 2)
    s["dx"][:n] = dx.reshape(-1, c["H"])[place].to(s["dx"].dtype)
    xt = x.transpose(1, 2)
    s["dgate"].copy_(xt @ dg)
    s["dup"].copy_(xt @ du)
    s["ddown"].copy_((g * sig * u).transpose(1, 2) @ dy)
    return {"dx": s["dx"], "dgate": s["dgate"], "dup": s["dup"], "ddown": s["ddown"]}


def plain_combine_backward(s):
    slot = s["pair_slot"].long()
    here = slot >= 0
    dy = s["dy"].float()
    s["dw"].copy_(torch.where(here, (s["y_perm"][slot.clamp(min=0)].float() * dy[:, None, :]).sum(2), 0.0))
    rows = (s["w"][:, :, None] * dy[:, None, :])[here]
    s["dy_perm"][slot[here]] = rows.to(s["dy_perm"].dtype)
    return {"dy_perm": s["dy_perm"], "dw": s["dw"]}


def plain_adamw(s):
    b1, b2 = s["b1"], s["b2"]
    q8 = s["case"]["state"] == "q8"
    g = [t.float() for t in s["g"]] if s["scale"] is None else [t.float() * s["scale"] for t in s["g"]]
    m = [dequantised(*t) for t in zip(s["m"], s["ms"])] if q8 else s["m"]
    v = [dequantised(*t).square() for t in zip(s["r"], s["rs"])] if q8 else s["v"]
    m = torch._foreach_add(torch._foreach_mul(m, b1), torch._foreach_mul(g, 1.0 - b1))
    v = torch._foreach_add(torch._foreach_mul(v, b2), torch._foreach_mul(torch._foreach_mul(g, g), 1.0 - b2))
    r = torch._foreach_sqrt(v)
    low = torch._foreach_add(torch._foreach_mul(r, 1.0 / math.sqrt(1.0 - b2 ** s["step"])), s["eps"])
    w = s["master"] or [t.float() for t in s["p"]]
    move = torch._foreach_mul(torch._foreach_div(m, low), s["lr"] / (1.0 - b1 ** s["step"]))
    w = torch._foreach_sub(torch._foreach_mul(w, 1.0 - s["lr"] * s["wd"]), move)
    torch._foreach_copy_(s["p"], w)
    if s["master"]:
        torch._foreach_copy_(s["master"], w)
    if q8:
        bits = [dither(t.numel(), s["seed"], s["step"]) for t in m]
        m, ms = zip(*[quantised(t, x >> 12) for t, x in zip(m, bits)])
        r, rs = zip(*[quantised(t, x & 0xFFFFF) for t, x in zip(r, bits)])
        [a.copy_(b) for a, b in zip(s["m"] + s["ms"] + s["r"] + s["rs"], m + ms + r + rs)]
    else:
        torch._foreach_copy_(s["m"], m)
        torch._foreach_copy_(s["v"], v)
    return adam_outputs(s)


def adam_outputs(s):
    return {name: s[name] for name in ("p", "master", "m", "ms", "v", "r", "rs") if name in s}


# ------------------------------------------------------------------------------------------------
# one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"ffn": own_ffn, "ffn_backward": own_ffn_backward, "combine_backward": own_combine_backward,
                "adamw": own_adamw}[op](state)
    return {"ffn": plain_ffn, "ffn_backward": plain_ffn_backward, "combine_backward": plain_combine_backward,
            "adamw": plain_adamw}[op](state)


def own_shape(s):
    """The shape, and for the block the workspace, that a program makes once and keeps."""
    from expert_ffn_layer_amd import native as N
    if "shape" not in s:
        c = s["case"]
        s["shape"] = N.make_shape(c["T"], c["H"], c.get("E", c["k"]), c["k"], c.get("I", 128), act=c["act"], w_routed=c["act"])
        if "E" in c:
            s["ws"] = torch.empty(N.moe_train_workspace_size(s["shape"]), dtype=torch.uint8, device=DEV)
            s["weights"] = {n: s[n] for n in ("gate", "up", "down")}
            s["groups"] = (s["off"], s["slot"]) if c["E"] > 1 else (None, None)
    return N


def own_ffn(s):
    N = own_shape(s)
    N.moe_gated_ffn(s["shape"], s["x"], *s["groups"], s["weights"], s["g"], s["u"], s["y"], s["ws"])
    return {"y": s["y"], "g": s["g"], "u": s["u"]}


def own_ffn_backward(s):
    N = own_shape(s)
    grads = {"gate": s["dgate"], "up": s["dup"], "down": s["ddown"]}
    N.moe_gated_ffn_backward(s["shape"], s["x"], *s["groups"], s["weights"], s["g"], s["u"], s["dy"], s["dx"], grads, s["ws"])
    return {"dx": s["dx"], "dgate": s["dgate"], "dup": s["dup"], "ddown": s["ddown"]}


def own_combine_backward(s):
    N = own_shape(s)
    N.moe_combine_backward(s["shape"], s["dy"], s["y_perm"], s["pair_slot"], s["w"], s["dy_perm"], s["dw"])
    return {"dy_perm": s["dy_perm"], "dw": s["dw"]}


def own_adamw(s):
    from expert_ffn_layer_amd import native as N
    if "table" not in s:
        q8 = s["case"]["state"] == "q8"
        s["table"] = N.adamw_tensors(s["p"], s["g"], s["m"], s["r" if q8 else "v"], s["master"] or None,
                                     s["ms"] if q8 else None, s["rs"] if q8 else None)
    N.moe_adamw(s["table"], lr=s["lr"], beta1=s["b1"], beta2=s["b2"], eps=s["eps"], weight_decay=s["wd"], step=s["step"],
                grad_scale=s["scale"], seed=s.get("seed", 0))
    return adam_outputs(s)


# ------------------------------------------------------------------------------------------------
# the least work of one pass

def work(case):
    c = case
    if c["op"] == "adamw":
        n, size = sum(tensor_sizes(c["sizes"])), {"f32": 4, "bf16": 2}
        each = size[c["g"]] + (8 + size[c["p"]] if c["master"] else 2 * size[c["p"]])
        each += 16 if c["state"] == "f32" else 4 + 16.0 / BLOCK
        return {"bytes": n * each, "flops": 16 * n}
    b = 4 if c["act"] == "f32" else 2
    T, H, k = c["T"], c["H"], c["k"]
    P = int(round(T * k * (1.0 - c["skip"])))
    if c["op"] == "combine_backward":
        return {"bytes": (T * H + 2 * P * H) * b + T * k * 12, "flops": 3 * P * H}
    E, I = min(c["E"], max(1, P)), c["I"]
    if c["op"] == "ffn":
        return {"bytes": (3 * E * H * I + T * H + P * H + 2 * P * I) * b, "flops": 6 * P * H * I}
    return {"bytes": (3 * (E + c["E"]) * H * I + T * H + 2 * P * H + 2 * P * I) * b, "flops": 12 * P * H * I}


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"ffn": exact_ffn, "ffn_backward": exact_ffn_backward, "combine_backward": exact_combine_backward,
            "adamw": exact_adamw}[case["op"]](s)


def exact_ffn(s):
    out = {name: torch.zeros(s[name].shape, dtype=torch.float64, device=DEV) for name in ("y", "g", "u")}
    ends = s["off"].tolist()
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        if a == b:
            continue
        x = s["x"].index_select(0, s["slot"][a:b].long()).double()
        out["g"][a:b] = torch.mm(x, s["gate"][e].double())
        out["u"][a:b] = torch.mm(x, s["up"][e].double())
        out["y"][a:b] = torch.mm(out["g"][a:b] * torch.sigmoid(out["g"][a:b]) * out["u"][a:b], s["down"][e].double())
    return out


def exact_ffn_backward(s):
    out = {name: torch.zeros(s[name].shape, dtype=torch.float64, device=DEV) for name in ("dx", "dgate", "dup", "ddown")}
    ends = s["off"].tolist()
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        if a == b:
            continue
        x = s["x"].index_select(0, s["slot"][a:b].long()).double()
        g, u, dy = s["g"][a:b].double(), s["u"][a:b].double(), s["dy"][a:b].double()
        gate, up, down = s["gate"][e].double(), s["up"][e].double(), s["down"][e].double()
        sig = torch.sigmoid(g)
        silu = g * sig
        dh = torch.mm(down, dy.t()).t()
        du = dh * silu
        dg = dh * u * (sig + silu * (1 - sig))
        out["dx"][a:b] = torch.mm(gate, dg.t()).t() + torch.mm(up, du.t()).t()
        out["dgate"][e], out["dup"][e] = torch.mm(x.t(), dg), torch.mm(x.t(), du)
        out["ddown"][e] = torch.mm((silu * u).t(), dy)
    return out


def exact_combine_backward(s):
    T, k = s["w"].shape
    dy = s["dy"].double()
    rows = torch.zeros(s["y_perm"].shape, dtype=torch.float64, device=DEV)
    dw = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    for j in range(k):
        slot = s["pair_slot"][:, j].long()
        t = torch.nonzero(slot >= 0).flatten()
        rows[slot[t]] = dy[t] * s["w"][t, j, None].double()
        dw[t, j] = torch.linalg.vecdot(dy[t], s["y_perm"][slot[t]].double())
    return {"dy_perm": rows, "dw": dw}


def random_words(n, seed, step):
    """The dither's definition on unsigned 32-bit words, by 16-bit halves that 64 bits hold exactly."""
    word = 1 << 32

    def times(x, c):
        return (x * (c % 65536) + (x * (c // 65536) % 65536) * 65536) % word

    key = (seed + step * 2654435769) % word
    key = (key ^ (key // 65536)) * 2246822519 % word
    key ^= key // 8192
    x = (times(torch.arange(n, device=DEV), 2654435761) + key) % word
    x = times(x ^ (x // 32768), 2246822519)
    return x ^ (x // 8192)


def e4m3(y, place):
    """The e4m3 value next below y, or above it where y's place between the two is past 1 - place: 3 bits below
    the leading one, a grid of 2^-9 under 2^-6, at most 448."""
    a = y.abs().clamp(max=448)
    grid = torch.ldexp(torch.ones_like(a), torch.frexp(a.clamp(min=2.0 ** -6))[1].sub(4))
    return torch.sign(y) * torch.floor(a / grid + place) * grid


def exact_adamw(s):
    scale = 1.0 if s["scale"] is None else s["scale"].double()
    q8 = s["case"]["state"] == "q8"
    out = {name: [] for name in adam_outputs(s)}
    for i, p in enumerate(s["p"]):
        g = s["g"][i].double() * scale
        if q8:
            block = torch.arange(g.numel(), device=DEV) // BLOCK
            m0, r0 = s["m"][i].double() * s["ms"][i].double()[block], s["r"][i].double() * s["rs"][i].double()[block]
            v0 = r0 * r0
        else:
            m0, v0 = s["m"][i].double(), s["v"][i].double()
        m, v = s["b1"] * m0 + (1 - s["b1"]) * g, s["b2"] * v0 + (1 - s["b2"]) * g * g
        mhat, vhat = m / (1 - s["b1"] ** s["step"]), v / (1 - s["b2"] ** s["step"])
        w0 = (s["master"][i] if s["master"] else p).double()
        w = w0 - s["lr"] * s["wd"] * w0 - s["lr"] * mhat / (vhat.sqrt() + s["eps"])
        out["p"].append(w)
        if s["master"]:
            out["master"].append(w)
        if not q8:
            out["m"].append(m)
            out["v"].append(v)
            continue
        words = random_words(g.numel(), s["seed"], s["step"])
        for name, t, bits in (("m", m, words // 4096), ("r", v.sqrt(), words % 1048576)):
            top = torch.zeros(s[name + "s"][i].numel(), dtype=torch.float64, device=DEV)
            top.scatter_reduce_(0, block, t.abs(), "amax").clamp_(min=2.0 ** -100)
            out[name].append(e4m3(t * 448 / top[block], bits.double() / 1048576))
            out[name + "s"].append(top / 448)
    return out
