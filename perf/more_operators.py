"""What today's recipes add to routing and training one MoE expert-FFN layer: the gate that picks experts by softmax or
sigmoid scores with a balancing bias and groups, its gradient, the orthogonalisation of matrices by Newton-Schulz
products, and the Muon step built on it.

``own`` chooses between the framework's entry points and the same operators in elementary torch operations."""
import math

import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
INF = float("inf")
NS = (3.4445, -4.7750, 2.0315)  # of the odd polynomial a s + b s^3 + c s^5 that a step applies to the singular values
STEPS, EPS = 5, 1e-7


# ------------------------------------------------------------------------------------------------
# cases

def gate(name, op, T, E, k, score, groups=1, top_groups=1, group_top=1, bias=False, renorm=True, scale=1.0, masked=0.0,
         padded=0.0):
    c = {"op": op, "T": T, "E": E, "k": k, "score": score, "groups": groups, "top_groups": top_groups,
         "group_top": group_top, "bias": bias, "renorm": renorm, "scale": scale, "masked": masked, "padded": padded}
    return {"name": name, **c} if name else c


def ortho(name, count, rows, cols, kind="bf16", rank=16):
    c = {"op": "orthogonalize", "count": count, "rows": rows, "cols": cols, "type": kind, "rank": rank}
    return {"name": name, **c} if name else c


def muon(name, stacks, p="bf16", master=False, nesterov=True, rank=16):
    c = {"op": "muon", "stacks": stacks, "p": p, "master": master, "nesterov": nesterov, "rank": rank}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one token of a decoding stream through a 256-expert gate with groups: launch latency counts
        gate("gate one token", "gate", 1, 256, 8, "sigmoid", 8, 4, 2, bias=True, scale=2.5),
        # an odd decode batch of a 128-expert softmax layer
        gate("gate softmax", "gate", 257, 128, 8, "softmax"),
        # a prefill chunk of a 384-expert layer without groups; experts of absent GPUs off, some rows padding
        gate("gate masked", "gate", 4099, 384, 6, "sigmoid", bias=True, scale=2.5, masked=0.1, padded=0.05),
        # the 16384-token batch of the 256-expert layer
        gate("gate grouped", "gate", 16384, 256, 8, "sigmoid", 8, 4, 2, bias=True, scale=2.5),
        # the gradient of a small softmax gate that keeps the probabilities as they are: every logit has one
        gate("gate backward softmax", "gate_backward", 333, 128, 4, "softmax", renorm=False),
        # the gradient of the 16384-token batch
        gate("gate backward grouped", "gate_backward", 16384, 256, 8, "sigmoid", 8, 4, 2, bias=True, scale=2.5),
        # the tiny fp32 layer's gate matrices: what a user's check runs
        ortho("orthogonalize tiny f32", 8, 256, 128, "f32"),
        # matrices of no round size, wide
        ortho("orthogonalize odd", 3, 771, 1000),
        # one matrix of the V3 layer alone (a shared expert's): few tiles for the whole card
        ortho("orthogonalize one", 1, 7168, 2048, rank=64),
        # every expert matrix and the router of the tiny fp32 layer
        muon("muon tiny f32", "8x256x128,8x256x128,8x128x256,1x256x8", "f32"),
        # a Qwen3-shaped slice of 16 experts in bf16
        muon("muon bf16", "16x4096x1536,16x4096x1536,16x1536x4096"),
        # a 32-expert slice of the V3 layer with fp32 master weights: the bulk of a training step's update
        muon("muon master", "32x7168x2048,32x7168x2048,32x2048x7168", master=True, rank=64),
    ]


def spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "gate", "gate", "gate_backward", "gate_backward", "orthogonalize", "orthogonalize", "muon"])
    if op in ("gate", "gate_backward"):
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        E = groups * spread(rng, max(2, 8 // groups), 1024 // groups)
        k = rng.randint(1, min(16, E))
        top = rng.randint(-(-k * groups // E), groups)
        T = min(spread(rng, 1, 16384), 16384 * 256 // E)
        # one renormalised weight is the scale whatever the logits
        return gate(None, op, T, E, k, rng.choice(["sigmoid", "softmax"]), groups, top, rng.choice([1, 2]),
                    rng.random() < 0.6, k > 1 and rng.random() < 0.7, rng.choice([1.0, 2.5]),
                    rng.choice([0.0, 0.0, 0.1]) if T > 32 else 0.0, rng.choice([0.0, 0.0, 0.1]) if T > 32 else 0.0)
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op == "orthogonalize":
        count, rows, cols = spread(rng, 1, 24), spread(rng, 8, 7168), spread(rng, 8, 7168)
        while cost(count, rows, cols) > (8e12 if kind == "bf16" else 1e12):
            count, rows = max(1, count // 2), rows * 3 // 4
        return ortho(None, count, rows, cols, kind, rng.randint(1, 32))
    E, H, I = spread(rng, 1, 16), 128 * spread(rng, 1, 32), 128 * spread(rng, 1, 16)
    while 3 * cost(E, H, I) > (16e12 if kind == "bf16" else 2e12):
        E, H = max(1, E // 2), max(128, H // 256 * 128)
    return muon(None, "%dx%dx%d,%dx%dx%d,%dx%dx%d,1x%dx%d" % (E, H, I, E, H, I, E, I, H, H, E), kind,
                kind == "bf16" and rng.random() < 0.5, rng.random() < 0.7, rng.randint(1, 32))


def sizes_of(text):
    return [tuple(int(n) for n in part.split("x")) for part in text.split(",")]


# ------------------------------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if case["op"] in ("gate", "gate_backward"):
        return prepare_gate(case, gen)
    if case["op"] == "orthogonalize":
        c = case
        g = gradient(gen, c["count"], c["rows"], c["cols"], c["rank"], 1.0).to(DT[c["type"]])
        return {"case": c, "g": g, "o": torch.zeros_like(g)}
    s = {"case": case, "lr": 1e-4, "momentum": 0.95, "wd": 0.1}
    sizes = sizes_of(case["stacks"])
    dt = DT[case["p"]]
    w = [torch.randn(z, device=DEV, generator=gen) * 0.02 for z in sizes]
    s["p"], s["master"] = [t.to(dt) for t in w], w if case["master"] else []
    s["g"] = [gradient(gen, *z, case["rank"], 1e-3).to(dt) for z in sizes]
    s["m"] = [gradient(gen, *z, case["rank"], 1e-2) for z in sizes]
    return s


def gradient(gen, count, rows, cols, rank, size):
    """Matrices as gradients are: some directions that many tokens share, of falling strength, over the noise of the rest."""
    r = min(rank, rows, cols)
    left = torch.randn(count, rows, r, device=DEV, generator=gen)
    left /= torch.arange(1, r + 1, device=DEV).sqrt()
    out = torch.bmm(left, torch.randn(count, r, cols, device=DEV, generator=gen))
    return out.add_(torch.randn(count, rows, cols, device=DEV, generator=gen)).mul_(size)


def prepare_gate(c, gen):
    """Logits of a trained router (some experts ask for more tokens than others), those of absent experts and of
    padding rows -inf; the bias against the experts' popularity; the gradient of the weights."""
    T, E, k = c["T"], c["E"], c["k"]
    popular = torch.randn(E, device=DEV, generator=gen) * 0.5
    logits = torch.randn(T, E, device=DEV, generator=gen) * 1.5 + popular
    logits[torch.rand(T, E, device=DEV, generator=gen) < c["masked"]] = -INF
    logits[torch.rand(T, device=DEV, generator=gen) < c["padded"]] = -INF
    s = {"case": c, "logits": logits, "bias": None}
    if c["bias"]:
        s["bias"] = torch.randn(E, device=DEV, generator=gen) * 0.02 - popular * 0.1
    s["idx"] = torch.zeros(T, k, dtype=torch.int32, device=DEV)
    s["w"] = torch.zeros(T, k, device=DEV)
    if c["op"] == "gate_backward":
        plain_gate(s)
        s["dw"] = torch.randn(T, k, device=DEV, generator=gen) * 0.1
        s["dlogits"] = torch.zeros(T, E, device=DEV)
    return s


# ------------------------------------------------------------------------------------------------
# plain forms

def scores(s):
    """The experts' scores in 64 bits (what is next to a border has to be told apart) and which of them may be chosen."""
    l = s["logits"].double()
    on = l > -INF
    if s["case"]["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l)), on
    e = torch.exp(l - torch.where(on, l, -1e300).amax(1, keepdim=True))
    e = torch.where(on, e, 0.0)
    return e / e.sum(1, keepdim=True).clamp(min=1e-300), on


def plain_gate(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    score, on = scores(s)
    choice = torch.where(on, score if s["bias"] is None else score + s["bias"].double(), -INF)
    if G > 1:
        best = torch.sort(choice.reshape(T, G, E // G), dim=2, descending=True).values[:, :, :2]
        value = best[:, :, 0]
        if c["group_top"] == 2 and E // G > 1:
            value = value + torch.where(best[:, :, 1] > -INF, best[:, :, 1], 0.0)
        kept = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        stays = torch.zeros(T, G, dtype=torch.bool, device=DEV).scatter_(1, kept, True)
        choice = torch.where(stays.repeat_interleave(E // G, dim=1), choice, -INF)
    value, order = torch.sort(choice, dim=1, descending=True, stable=True)
    idx = torch.where(value[:, :k] > -INF, order[:, :k], E).sort(dim=1).values
    here = idx < E
    w = torch.where(here, score.gather(1, idx.clamp(max=E - 1)), 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    s["idx"].copy_(torch.where(here, idx, -1))
    s["w"].copy_(w * c["scale"])
    return {"idx": s["idx"], "w": s["w"]}


def plain_gate_backward(s):
    c = s["case"]
    score, on = scores(s)
    here = s["idx"] >= 0
    at = s["idx"].clamp(min=0).long()
    chosen = torch.where(here, score.gather(1, at), 0.0)
    dw = torch.where(here, s["dw"].double(), 0.0) * c["scale"]
    if c["renorm"]:
        total = chosen.sum(1, keepdim=True).clamp(min=1e-300)
        dw = (dw - (dw * chosen).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(score).scatter_add_(1, at, torch.where(here, dw, 0.0))
    if c["score"] == "sigmoid":
        d = ds * score * (1.0 - score)
    else:
        d = score * (ds - (ds * score).sum(1, keepdim=True))
    s["dlogits"].copy_(torch.where(on, d, 0.0))
    return s["dlogits"]


def newton_schulz(u):
    """The last axes' matrices with their singular values brought near 1, in 32 bits."""
    norm = u.square().sum((1, 2), keepdim=True, dtype=torch.float64).sqrt()
    x = (u / (norm + EPS)).float()
    a, b, c = NS
    wide = u.shape[1] <= u.shape[2]
    for _ in range(STEPS):
        xt = x.transpose(1, 2)
        gram = torch.bmm(x, xt) if wide else torch.bmm(xt, x)
        poly = b * gram + c * torch.bmm(gram, gram)
        x = a * x + (torch.bmm(poly, x) if wide else torch.bmm(x, poly))
    return x


def plain_orthogonalize(s):
    s["o"].copy_(newton_schulz(s["g"].float()))
    return s["o"]


def plain_muon_stack(s, i):
    mu, lr = s["momentum"], s["lr"]
    g, m, p = s["g"][i].float(), s["m"][i], s["p"][i]
    m.copy_(mu * m + g)
    o = newton_schulz(g + mu * m if s["case"]["nesterov"] else m)
    w = s["master"][i] if s["master"] else p.float()
    w = w * (1.0 - lr * s["wd"]) - lr * 0.2 * math.sqrt(max(p.shape[1:])) * o
    p.copy_(w)
    if s["master"]:
        s["master"][i].copy_(w)


def plain_muon(s):
    [plain_muon_stack(s, i) for i in range(len(s["p"]))]
    return {name: s[name] for name in ("p", "m", "master")}


# ------------------------------------------------------------------------------------------------
# one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"gate": own_gate, "gate_backward": own_gate_backward, "orthogonalize": own_orthogonalize, "muon": own_muon}[op](state)
    return {"gate": plain_gate, "gate_backward": plain_gate_backward, "orthogonalize": plain_orthogonalize,
            "muon": plain_muon}[op](state)


def own_rule(s):
    """The shape and the rule that a program makes once and keeps."""
    from expert_ffn_layer_amd import native as N
    if "rule" not in s:
        c = s["case"]
        s["shape"] = N.make_shape(c["T"], 128, c["E"], c["k"], 128)
        s["rule"] = N.make_gate(c["score"], groups=c["groups"], top_groups=c["top_groups"], group_top=c["group_top"],
                                renormalize=c["renorm"], scale=c["scale"])
    return N


def own_gate(s):
    N = own_rule(s)
    N.moe_gate(s["shape"], s["rule"], s["logits"], s["bias"], s["idx"], s["w"])
    return {"idx": s["idx"], "w": s["w"]}


def own_gate_backward(s):
    N = own_rule(s)
    N.moe_gate_backward(s["shape"], s["rule"], s["logits"], s["idx"], s["dw"], s["dlogits"])
    return s["dlogits"]


def own_orthogonalize(s):
    from expert_ffn_layer_amd import native as N
    if "ws" not in s:
        s["ws"] = torch.empty(N.moe_orthogonalize_workspace_size(s["case"]["type"], *s["g"].shape), dtype=torch.uint8, device=DEV)
    N.moe_orthogonalize(s["g"], s["o"], s["ws"], steps=STEPS, coefficients=NS, eps=EPS)
    return s["o"]


def own_muon(s):
    from expert_ffn_layer_amd import native as N
    if "table" not in s:
        scale = [0.2 * math.sqrt(max(t.shape[1:])) for t in s["p"]]
        s["table"] = N.muon_tensors(s["p"], s["g"], s["m"], s["master"] or None, scale)
        s["ws"] = torch.empty(N.moe_muon_workspace_size(s["table"]), dtype=torch.uint8, device=DEV)
    N.moe_muon(s["table"], s["ws"], lr=s["lr"], momentum=s["momentum"], nesterov=s["case"]["nesterov"], weight_decay=s["wd"],
               steps=STEPS, coefficients=NS, eps=EPS)
    return {name: s[name] for name in ("p", "m", "master")}


# ------------------------------------------------------------------------------------------------
# the least work of one pass

def cost(count, rows, cols):
    """Operations of the steps: the products with a symmetric result take one half of it."""
    m, n = min(rows, cols), max(rows, cols)
    return float(STEPS * count) * (3.0 * m * m * n + float(m) ** 3)


def work(case):
    c = case
    if c["op"] in ("gate", "gate_backward"):
        T, E, k = c["T"], c["E"], c["k"]
        if c["op"] == "gate":
            return {"bytes": 4 * T * E + 8 * T * k + (4 * E if c["bias"] else 0), "flops": 4 * T * E}
        every = c["score"] == "softmax" and not c["renorm"]
        return {"bytes": 4 * T * E + 8 * T * k + 4 * T * (E if every else k), "flops": 2 * T * E if every else 8 * T * k}
    size = {"f32": 4, "bf16": 2}
    if c["op"] == "orthogonalize":
        n = c["count"] * c["rows"] * c["cols"]
        return {"bytes": 2 * n * size[c["type"]], "flops": cost(c["count"], c["rows"], c["cols"])}
    sizes = sizes_of(c["stacks"])
    n = sum(a * b * d for a, b, d in sizes)
    each = size[c["p"]] + 8 + (8 + size[c["p"]] if c["master"] else 2 * size[c["p"]])
    return {"bytes": n * each, "flops": sum(cost(*z) for z in sizes)}


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"gate": exact_gate, "gate_backward": exact_gate_backward, "orthogonalize": exact_orthogonalize,
            "muon": exact_muon}[case["op"]](s)


def exact_scores(s):
    l = s["logits"].double()
    if s["case"]["score"] == "sigmoid":
        return torch.sigmoid(l)
    return torch.softmax(l, 1).nan_to_num(0.0)


def places(v):
    """How many come before each value of a row, larger ones and equal ones of lower index; rows in parts for memory."""
    before = torch.ones(v.shape[1], v.shape[1], dtype=torch.bool, device=DEV).tril(-1)
    out = []
    for part in v.split(max(1, (1 << 28) // v.shape[1] ** 2)):
        a, b = part[:, :, None], part[:, None, :]
        out.append(((b > a) | ((b == a) & before)).sum(2))
    return torch.cat(out)


def exact_gate(s):
    c = s["case"]
    T, E, G = c["T"], c["E"], c["groups"]
    p = exact_scores(s)
    v = p if s["bias"] is None else p + s["bias"].double()
    v = v.masked_fill(torch.isneginf(s["logits"]), -INF)
    if G > 1:
        top = v.reshape(T, G, -1).topk(min(c["group_top"], E // G), dim=2).values
        worth = top.nan_to_num(neginf=0.0).sum(2).masked_fill(torch.isneginf(top[:, :, 0]), -INF)
        out = (places(worth) >= c["top_groups"])[:, :, None].expand(T, G, E // G).reshape(T, E)
        v = v.masked_fill(out, -INF)
    taken = (places(v) < c["k"]) & ~torch.isneginf(v)
    w = p * taken
    if c["renorm"]:
        w = (w / w.sum(1, keepdim=True)).nan_to_num(0.0)
    # the taken ones to the front, in their order
    front = torch.sort(taken.to(torch.int8), dim=1, descending=True, stable=True)
    k = c["k"]
    return {"idx": torch.where(front.values[:, :k] > 0, front.indices[:, :k], -1).int(),
            "w": c["scale"] * w.gather(1, front.indices[:, :k])}


def exact_gate_backward(s):
    """By torch's own differentiation of the weights."""
    c = s["case"]
    l = s["logits"].double().masked_fill(torch.isneginf(s["logits"]), -800.0).requires_grad_()
    p = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
    here = s["idx"] >= 0
    w = p.gather(1, s["idx"].clamp(min=0).long()) * here
    if c["renorm"]:
        w = w / torch.where(here.any(1, keepdim=True), w.sum(1, keepdim=True), 1.0)
    (c["scale"] * w * s["dw"].double() * here).sum().backward()
    return l.grad.masked_fill(torch.isneginf(s["logits"]), 0.0)


def exact_newton_schulz(u):
    """One matrix: the polynomial in Gram's matrix by Horner's rule, the short side first."""
    a, b, c = NS
    x = u / (torch.linalg.matrix_norm(u) + EPS)
    x = x if u.shape[0] <= u.shape[1] else x.t().contiguous()
    one = torch.eye(x.shape[0], dtype=torch.float64, device=DEV)
    for _ in range(STEPS):
        gram = torch.mm(x, x.t())
        x = torch.mm(torch.mm(gram, c * gram + b * one) + a * one, x)
    return x if u.shape[0] <= u.shape[1] else x.t()


def exact_orthogonalize(s):
    return torch.stack([exact_newton_schulz(g.double()) for g in s["g"]])


def exact_muon(s):
    out = {"p": [], "m": [], "master": []}
    for i, p in enumerate(s["p"]):
        w = torch.empty(p.shape, dtype=torch.float64, device=DEV)
        m = s["momentum"] * s["m"][i].double() + s["g"][i].double()
        for e in range(p.shape[0]):
            u = s["g"][i][e].double() + s["momentum"] * m[e] if s["case"]["nesterov"] else m[e]
            old = (s["master"][i] if s["master"] else p)[e].double()
            w[e] = old - s["lr"] * (s["wd"] * old + 0.2 * math.sqrt(max(p.shape[1:])) * exact_newton_schulz(u))
        out["p"].append(w)
        out["m"].append(m)
        if s["master"]:
            out["master"].append(w)
    return out
