"""The gate and its gradient on the GPU against their 64-bit definitions."""
import math

import pytest
import torch

from expert_ffn_layer_amd import native as N

from _gpu import say
from _muon import F, gate_gradient, gate_row

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
INF = math.inf


def shape(T, E, k):
    return N.make_shape(T, 128, E, k, 128)


def rule(score="sigmoid", groups=1, top_groups=None, group_top=1, renormalize=True, scale=1.0):
    return dict(score=score, groups=groups, top_groups=groups if top_groups is None else top_groups, group_top=group_top,
                renormalize=renormalize, scale=scale)


def run(logits, bias, k, r):
    T, E = logits.shape
    idx = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T, k), 99.0, device=DEV)
    N.moe_gate(shape(T, E, k), N.make_gate(**r), logits.to(DEV), None if bias is None else bias.to(DEV), idx, w)
    return idx.cpu(), w.cpu()


def verify(logits, bias, k, r):
    idx, w = run(logits, bias, k, r)
    b = None if bias is None else bias.numpy()
    for t in range(logits.shape[0]):
        want, weights = gate_row(logits[t].numpy(), b, k, **r)
        assert idx[t].tolist() == want, "token %d: %s, not %s" % (t, idx[t].tolist(), want)
        assert all(abs(x - y) <= F * abs(y) + 2.0 ** -149 for x, y in zip(w[t].tolist(), weights)), "token %d: %s, not %s" % (t, w[t].tolist(), weights)
    return idx


def inputs(T, E, seed, masked=0.0, bias=True):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g) * 2
    logits[torch.rand(T, E, generator=g) < masked] = -INF
    return logits, torch.randn(E, generator=g) * 0.1 if bias else None


RULES = {
    "sigmoid": rule(),
    "sigmoid as it is": rule(renormalize=False, scale=2.5),
    "softmax": rule("softmax"),
    "softmax as it is": rule("softmax", renormalize=False, scale=0.5),
}
SIZES = [(1, 8, 1), (1, 1, 1), (3, 2, 2), (9, 63, 5), (5, 64, 8), (7, 65, 16), (4, 128, 8), (130, 192, 3), (3, 256, 8), (6, 384, 6),
         (2, 1000, 16), (5, 1024, 1)]


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("name", RULES)
@pytest.mark.parametrize("T,E,k", SIZES)
def test_gate(T, E, k, name, bias):
    say("gate", T, E, k, name, bias)
    logits, b = inputs(T, E, 100 * E + k, bias=bias)
    verify(logits, b, k, RULES[name])


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,groups,top_groups,group_top", [
    (256, 8, 8, 4, 2), (256, 8, 8, 4, 1), (60, 5, 3, 1, 2), (60, 5, 3, 2, 1), (64, 16, 64, 16, 2), (64, 3, 64, 50, 1), (1024, 16, 16, 1, 2),
    (128, 8, 2, 1, 2), (8, 2, 4, 1, 2), (960, 9, 60, 7, 2), (1000, 10, 50, 20, 1)])
def test_groups(E, k, groups, top_groups, group_top, score, bias):
    say("groups", E, k, groups, top_groups, group_top, score, bias)
    logits, b = inputs(33, E, E + groups, bias=bias)
    verify(logits, b, k, rule(score, groups, top_groups, group_top))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (8, 3)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_experts_that_are_off(score, groups, top_groups, renormalize):
    """Rows with few experts, one, and none; groups with one and none; experts off by their bias."""
    T, E, k = 40, 64, 6
    logits, b = inputs(T, E, 5, masked=0.6)
    logits[3] = -INF
    logits[4, 1:] = -INF
    logits[5, :60] = -INF
    for t in range(6, 12):  # one expert in every group, or in some
        keep = logits[t, ::8].clone()
        logits[t] = -INF
        logits[t, ::8] = keep
    b[::7] = -INF
    r = rule(score, groups, top_groups, 2, renormalize, 2.0)
    idx = verify(logits, b, k, r)
    assert (idx[3] == -1).all() and (idx[:, 1:] == -1).any()
    verify(logits, None, k, r)


def test_equal_choices_go_to_the_lower_index():
    T, E, k = 5, 256, 8
    logits = torch.zeros(T, E)
    logits[1, 100:] = 1.0
    logits[2] = torch.arange(E) % 5
    logits[3, ::2] = -0.0
    logits[4] = torch.where(torch.arange(E) < 128, 1.0, 1.0)
    bias = torch.zeros(E)
    for b in (None, bias):
        for r in (rule(), rule("softmax"), rule(groups=8, top_groups=2, group_top=2), rule("softmax", 8, 3, 1)):
            verify(logits, b, k, r)
    # what the bias takes from one it gives to the other: 2^-3 in both places
    logits = torch.zeros(1, 4)
    verify(logits, torch.tensor([0.125, 0.25, 0.25, 0.125]), 2, rule())


def test_a_border_that_32_bits_do_not_see():
    """Sigmoids of neighbouring logits near 6 are 1.2e-9 apart, an fp32 step there is 6e-8."""
    E, k = 256, 1
    x = torch.tensor(6.0)
    up = torch.nextafter(x, torch.tensor(10.0))
    logits = torch.zeros(4, E)
    for t, e in enumerate((1, 63, 64, 255)):
        logits[t, 0], logits[t, e] = x, up
    for b in (torch.zeros(E), torch.full((E,), 0.3)):
        idx = verify(logits, b, k, rule(scale=1.5))
        assert idx.flatten().tolist() == [1, 63, 64, 255]
    # and a group that is best by as little
    verify(logits, torch.zeros(E), k, rule(groups=4, top_groups=1, group_top=2))
    verify(logits, torch.zeros(E), k, rule("softmax", groups=4, top_groups=1, group_top=2))


@pytest.mark.parametrize("E,k,groups,top_groups", [(64, 6, 1, 1), (256, 8, 8, 4), (300, 8, 4, 2), (768, 16, 1, 1)])
def test_many_tokens_with_borders_that_32_bits_do_not_see(E, k, groups, top_groups):
    """Some tokens have 2 to 24 experts within 2e-8 of each other around the last chosen, some of them equal."""
    g = torch.Generator().manual_seed(E)
    T = 2300
    logits = torch.randn(T, E, generator=g)
    bias = torch.rand(E, generator=g) * 2.0 ** -30  # keeps the order of the sigmoids below in doubt, not what is far
    steps = torch.tensor([6.0 + i * 2.0 ** -21 for i in range(6)])
    for t in range(0, T, 3):
        n = int(torch.randint(2, 25, (1,), generator=g))
        few = torch.randperm(E, generator=g)[:n + k // 2]
        logits[t, few[:n]] = steps[torch.randint(0, 6, (n,), generator=g)]
        logits[t, few[n:]] = 8.0 + torch.rand(len(few) - n, generator=g)
    for b in (bias, torch.zeros(E)):
        verify(logits, b, k, rule(groups=groups, top_groups=top_groups, group_top=2, scale=1.5))


def test_far_logits():
    """Weights that are renormalised keep their ratios where the scores themselves vanish."""
    logits = torch.tensor([[-200.0, -201.0, -300.0, -1e30], [90.0, 91.0, 100.0, 1e30], [-90.0, 80.0, 0.0, -100.0],
                           [3e38, -3e38, 1.0, 2.0], [-1e38, -2e38, -3e38, -3.3e38]])
    idx, w = run(logits, None, 3, rule())
    assert idx.tolist() == [[0, 1, 2], [1, 2, 3], [0, 1, 2], [0, 2, 3], [0, 1, 2]]
    e = math.exp(-1.0)
    assert abs(w[0, 0] - 1 / (1 + e)) < 1e-6 and abs(w[0, 1] - e / (1 + e)) < 1e-6 and w[0, 2] < 1e-40
    assert torch.allclose(w[1], torch.tensor([1 / 3] * 3)) and torch.isfinite(w).all()
    assert w[4].tolist() == [1.0, 0.0, 0.0]
    verify(logits, None, 4, rule("softmax"))
    verify(logits, None, 2, rule("softmax", renormalize=False))


def test_nan_and_infinity():
    logits, b = inputs(6, 64, 9)
    logits[1, 40] = math.nan
    logits[2, 7] = INF
    logits[3] = math.nan
    clean = [0, 4, 5]
    for r in (rule(), rule("softmax"), rule(renormalize=False), rule(groups=4, top_groups=2, group_top=2), rule("softmax", 4, 1, 1, False)):
        for bias in (None, b):
            idx, w = run(logits, bias, 4, r)
            if r["score"] == "sigmoid":  # in a softmax every score is NaN
                assert 40 in idx[1].tolist() and w[1, idx[1].tolist().index(40)].isnan()
            assert (w[1].isnan().all()) == (r["score"] == "softmax" or r["renormalize"])
            assert idx[3].tolist() == [0, 1, 2, 3] and w[3].isnan().all()
            if r["score"] == "sigmoid":
                verify(logits[2:3], bias, 4, r)
            else:
                assert w[2].isnan().any()
            for t in clean:  # other rows do not change
                assert idx[t].tolist() == gate_row(logits[t].numpy(), None if bias is None else bias.numpy(), 4, **r)[0]
    bias = b.clone()
    bias[9] = math.nan
    idx, w = run(logits[clean], bias, 4, rule())
    assert (idx == 9).any(1).all() and torch.isfinite(w).all()  # the largest choice; no bias in the weights


@pytest.mark.parametrize("masked", [0.0, 0.4])
@pytest.mark.parametrize("name", RULES)
@pytest.mark.parametrize("T,E,k", SIZES)
def test_gradient(T, E, k, name, masked):
    say("gate gradient", T, E, k, name, masked)
    r = RULES[name]
    logits, _ = inputs(T, E, E + 7 * k, masked)
    idx, _ = run(logits, None, k, r)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(k))
    got = torch.full((T, E), 77.0, device=DEV)
    args = [t.to(DEV) for t in (logits, idx, dw)]
    N.moe_gate_backward(shape(T, E, k), N.make_gate(**r), *args, got)
    want, bound = gate_gradient(logits, idx, dw, r["score"], r["renormalize"], r["scale"])
    assert ((got.cpu().double() - want).abs() <= bound + 2.0 ** -149).all()
    N.moe_gate_backward(shape(T, E, k), N.make_gate(**r), *args, args[0])  # into the logits' memory
    assert torch.equal(args[0], got)


@pytest.mark.parametrize("name", RULES)
def test_gradient_against_differences(name):
    """Of the definition's weights: (w(l + h) - w(l - h)) / 2h, off by h^2/6 times a third derivative of at most 2 scale |dw|."""
    r, T, E, k, h = RULES[name], 3, 24, 4, 1e-4
    logits, b = inputs(T, E, 3)
    idx, _ = run(logits, b, k, r)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(1))
    got = torch.empty(T, E, device=DEV)
    N.moe_gate_backward(shape(T, E, k), N.make_gate(**r), logits.to(DEV), idx.to(DEV), dw.to(DEV), got)

    def value(l):
        s = torch.sigmoid(l) if r["score"] == "sigmoid" else torch.softmax(l, 1)
        w = s.gather(1, idx.long())
        if r["renormalize"]:
            w = w / w.sum(1, keepdim=True)
        return float((r["scale"] * w * dw.double()).sum())
    for t in range(T):
        for e in range(E):
            step = torch.zeros(T, E, dtype=torch.float64)
            step[t, e] = h
            want = (value(logits.double() + step) - value(logits.double() - step)) / (2 * h)
            most = float(dw[t].abs().sum()) * abs(r["scale"])
            assert abs(float(got[t, e]) - want) <= most * (h * h / 3 + F) + 1e-10


def test_gradient_of_rows_that_the_gate_does_not_make():
    """The same expert twice adds up; experts out of range and off take no part; their gradients are not read."""
    T, E = 3, 70
    logits, _ = inputs(T, E, 4)
    logits[1, 5] = -INF
    idx = torch.tensor([[3, 3, 69, 8], [5, 70, -9, 12], [-1, -1, -1, 1 << 30]], dtype=torch.int32)
    dw = torch.tensor([[1.0, -2.0, 0.5, 3.0], [math.nan, math.nan, math.nan, 2.0], [math.nan] * 4])
    for r in RULES.values():
        got = torch.full((T, E), 77.0, device=DEV)
        N.moe_gate_backward(shape(T, E, 4), N.make_gate(**r), logits.to(DEV), idx.to(DEV), dw.to(DEV), got)
        want, bound = gate_gradient(logits, idx, dw, r["score"], r["renormalize"], r["scale"])
        assert ((got.cpu().double() - want).abs() <= bound + 2.0 ** -149).all()
        assert (got[2] == 0).all()


def test_many_tokens_and_no_tokens():
    T, E, k = 70001, 40, 3
    logits = torch.randn(T, E, device=DEV, generator=torch.Generator(device=DEV).manual_seed(2))
    idx, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    N.moe_gate(shape(T, E, k), N.make_gate("sigmoid"), logits, None, idx, w)
    want = logits.topk(k, dim=1).indices.sort(dim=1).values
    assert torch.equal(idx.long(), want)
    s = torch.sigmoid(logits.double()).gather(1, want)
    assert ((w - s / s.sum(1, keepdim=True)).abs() <= F * w).all()
    none = torch.empty(0, E, device=DEV)
    N.moe_gate(shape(0, E, k), N.make_gate(), none, None, torch.empty(0, k, dtype=torch.int32, device=DEV), torch.empty(0, k, device=DEV))
    N.moe_gate_backward(shape(0, E, k), N.make_gate(), none, torch.empty(0, k, dtype=torch.int32, device=DEV), torch.empty(0, k, device=DEV), none.clone())


def test_captured_gate_and_gradient():
    """Replays follow the logits, with eager calls of other sizes between them."""
    T, E, k = 2500, 96, 6
    r = N.make_gate(**rule(groups=8, top_groups=3, group_top=2, scale=2.0))
    s = shape(T, E, k)
    logits, bias = (t.to(DEV) for t in inputs(T, E, 5))
    dw = torch.randn(T, k, device=DEV)
    idx, w, d = (torch.empty(n, dtype=t, device=DEV) for n, t in (((T, k), torch.int32), ((T, k), torch.float32), ((T, E), torch.float32)))

    def both(l, i, w, d):
        N.moe_gate(s, r, l, bias, i, w)
        N.moe_gate_backward(s, r, l, i, dw, d)
    both(logits, idx, w, d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(logits, idx, w, d)
    for i in range(4):
        logits.copy_(torch.randn(T, E, device=DEV) * 2)
        graph.replay()
        other = [torch.empty_like(t) for t in (idx, w, d)]
        both(logits.clone(), *other)
        run(*inputs(7, 40, i), 4, rule())
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((idx, w, d), other)), "replay %d" % i


def test_gradient_in_the_logits_memory():
    for name in RULES:
        T, E, k = 1000, 200, 5
        r, s = N.make_gate(**RULES[name]), shape(T, E, k)
        logits, b = inputs(T, E, 9)
        idx, _ = run(logits, b, k, RULES[name])
        l, i, dw = logits.to(DEV), idx.to(DEV), torch.randn(T, k, device=DEV)
        d = torch.empty_like(l)
        N.moe_gate_backward(s, r, l, i, dw, d)
        N.moe_gate_backward(s, r, l, i, dw, l)
        assert torch.equal(d, l), name
