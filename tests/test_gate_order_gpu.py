"""The order in which the gate takes experts, where it is hard to tell, and the rounding of its numbers, on the GPU."""
import math

import pytest
import torch

from expert_ffn_layer_amd import native as N

from _gpu import say
from _muon import F

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
INF = math.inf


def shape(T, E, k):
    return N.make_shape(T, 128, E, k, 128)


def gate(logits, bias, k, rule):
    T, E = logits.shape
    idx = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T, k), 99.0, device=DEV)
    N.moe_gate(shape(T, E, k), rule, logits.to(DEV), None if bias is None else bias.to(DEV), idx, w)
    return idx.cpu().long(), w.cpu()


def by_logits(logits, k, groups, top_groups):
    """[T, k] experts in ascending order, E where there are fewer: groups by their largest logit, equal ones to the lower index."""
    T, E = logits.shape
    order = logits.double()
    if groups > 1:
        worth = order.reshape(T, groups, -1).amax(2)
        kept = worth.sort(dim=1, descending=True, stable=True).indices[:, :top_groups]
        stays = torch.zeros(T, groups, dtype=torch.bool).scatter_(1, kept, True)
        order = order.masked_fill(~stays.repeat_interleave(E // groups, 1), -INF)
    top = order.sort(dim=1, descending=True, stable=True)
    return torch.where(top.values[:, :k] > -INF, top.indices[:, :k], E).sort(1).values


def weights(logits, idx, score, renormalize, scale):
    """In 64 bits; a score that vanishes keeps its ratio to the others."""
    l = logits.double()
    here = idx < l.shape[1]
    v = torch.where(here, l.gather(1, idx.clamp(max=l.shape[1] - 1)), -INF)
    x = v.clamp(max=0.0) if score == "sigmoid" else v
    most = torch.zeros(len(l), 1, dtype=torch.float64)
    if renormalize:
        most = x.amax(1, keepdim=True)
    elif score == "softmax":
        most = l.amax(1, keepdim=True)
    most = torch.where(most > -INF, most, 0.0)
    s = torch.exp(x - most)
    if score == "sigmoid":
        s = s / (1.0 + torch.exp(-v.abs()))
    s = torch.where(here, s, 0.0)
    if renormalize:
        s = s / s.sum(1, keepdim=True).clamp(min=1e-300)
    elif score == "softmax":
        s = s / torch.exp(l - most).sum(1, keepdim=True).clamp(min=1e-300)
    return scale * s


LEVELS = [0.0, 40.0, 60.0, 800.0, -40.0, -790.0]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("E,k,groups,top_groups", [(3, 1, 1, 1), (4, 2, 1, 1), (40, 8, 1, 1), (256, 8, 1, 1), (256, 8, 8, 3), (300, 5, 4, 2),
                                                   (600, 16, 1, 1), (1024, 3, 64, 2), (60, 5, 3, 2)])
@pytest.mark.parametrize("T", [40, 2300])
def test_equal_logits_where_scores_saturate(T, E, k, groups, top_groups, score, renormalize):
    """Without a bias the logits are the order, whatever becomes of the scores: 1 or 0 in any number of bits, or past the
    exponential's range."""
    say("equal logits", T, E, k, groups, top_groups, score, renormalize)
    g = torch.Generator().manual_seed(E + T)
    logits = torch.randint(0, 6, (T, E), generator=g).float() + torch.tensor(LEVELS)[torch.arange(T) % len(LEVELS)][:, None]
    logits[::5][torch.rand(len(logits[::5]), E, generator=g) < 0.5] = -INF
    rule = N.make_gate(score, groups, top_groups, 1, renormalize, 1.5)
    idx, w = gate(logits, None, k, rule)
    want = by_logits(logits, k, groups, top_groups)
    assert torch.equal(torch.where(want < E, want, -1), idx)
    exact = weights(logits, want, score, renormalize, 1.5)
    assert ((w.double() - exact).abs() <= F * exact + 2.0 ** -149).all()


@pytest.mark.parametrize("l,k,experts", [([50.0, 60, 60], 1, [1]), ([38.0, 40, 40, 39], 2, [1, 2]), ([-800.0, -790, -790], 1, [1]), ([40.0, 41, 41], 1, [1]),
                                         ([50.0, 50, 40, 45], 3, [0, 1, 3])])
def test_a_few_equal_logits(l, k, experts):
    for score in ("sigmoid", "softmax"):
        idx, _ = gate(torch.tensor([l]), None, k, N.make_gate(score))
        assert idx.tolist() == [experts]
    idx, w = gate(torch.tensor([[800.0, 800, 1, 2], [-800.0, -800, -801, -900]]), None, 2, N.make_gate())
    assert idx.tolist() == [[0, 1], [0, 1]] and w.tolist() == [[0.5, 0.5]] * 2


def by_choices(logits, bias, k):
    """[T, k] experts in ascending order by sigmoid and bias in 64 bits, equal ones to the lower index."""
    c = 1.0 / (1.0 + torch.exp(-logits.double())) + bias.double()
    return c.sort(dim=1, descending=True, stable=True).indices[:, :k].sort(1).values


@pytest.mark.parametrize("T", [500, 2300])
@pytest.mark.parametrize("E,k", [(24, 3), (64, 6), (256, 8), (300, 16), (768, 6)])
def test_borders_among_equal_choices(T, E, k):
    """Choices spread over one to four times what fp32 tells apart, so that some are equal in fp32, above the border, on it and
    below, while others end just outside of what is looked at again."""
    say("borders", T, E, k)
    g = torch.Generator().manual_seed(E + T)
    bias = torch.randn(E, generator=g) * 0.2
    logits = torch.randn(T, E, generator=g) - 4.0
    for t in range(T):
        n = int(torch.randint(2, min(E, 25), (1,), generator=g))
        few = torch.randperm(E, generator=g)[:n + k // 3]
        width = 2.0 ** -float(torch.randint(19, 25, (1,), generator=g))
        want = 0.6 + width * torch.rand(len(few), generator=g, dtype=torch.float64)
        want[n:] += 0.1
        s = (want - bias[few].double()).clamp(0.01, 0.99)
        logits[t, few] = torch.log(s / (1.0 - s)).float()
    want = by_choices(logits, bias, k)
    idx, _ = gate(logits, bias, k, N.make_gate("sigmoid"))
    bad = (idx != want).any(1).nonzero().flatten().tolist()
    assert not bad, "%d tokens, the first %d: %s, not %s" % (len(bad), bad[0], idx[bad[0]].tolist(), want[bad[0]].tolist())


def test_a_border_two_equal_choices_deep():
    """The three equal choices went in one round, so that the border looked for lay below the fourth."""
    logits = torch.tensor([[0.0, 0.0, 0.0, 1.5563236, -30.0, -3.0]])
    bias = torch.tensor([-0.4, -0.4, -0.4, -0.7258252, 0.09999926, -1.0])
    want = by_choices(logits, bias, 3)
    assert want.tolist() == [[0, 1, 3]]
    for T in (1, 2500):
        idx, _ = gate(logits.expand(T, -1).contiguous(), bias, 3, N.make_gate("sigmoid"))
        assert (idx == want).all()


def by_groups(scores, bias, k, groups, top_groups):
    """The definition with sums of two in 64 bits, for groups of at least two that may all be chosen."""
    c = scores.double() + bias.double()
    worth = c.reshape(len(c), groups, -1).topk(2, dim=2).values.sum(2)
    kept = worth.sort(dim=1, descending=True, stable=True).indices[:, :top_groups]
    stays = torch.zeros(len(c), groups, dtype=torch.bool).scatter_(1, kept, True).repeat_interleave(c.shape[1] // groups, 1)
    return c.masked_fill(~stays, -INF).sort(dim=1, descending=True, stable=True).indices[:, :k].sort(1).values


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("size", [10.0, 100.0, 1000.0, 2e38])
@pytest.mark.parametrize("E,groups,top_groups,k", [(64, 8, 3, 5), (256, 8, 4, 8), (24, 2, 1, 3), (1024, 16, 7, 6), (120, 4, 2, 4)])
@pytest.mark.parametrize("T", [300, 2300])
def test_group_values_that_cancel(T, E, groups, top_groups, k, size, score):
    """Biases of one size and both signs in each group: its value is the small rest of two large numbers."""
    say("groups that cancel", T, E, groups, top_groups, k, size, score)
    g = torch.Generator().manual_seed(E)
    n = E // groups
    bias = torch.full((E,), -size)
    bias[torch.arange(groups) * n + torch.randint(0, n, (groups,), generator=g)] = size
    logits = torch.randn(T, E, generator=g) * 10.0 ** -torch.randint(0, 5, (T, 1), generator=g).float()
    logits = logits + torch.randn(T, 1, generator=g)
    s = torch.sigmoid(logits.double()) if score == "sigmoid" else torch.softmax(logits.double(), 1)
    want = by_groups(s, bias, k, groups, top_groups)
    idx, _ = gate(logits, bias, k, N.make_gate(score, groups, top_groups, 2))
    bad = (idx != want).any(1).nonzero().flatten().tolist()
    assert not bad, "%d tokens, the first %d: %s, not %s" % (len(bad), bad[0], idx[bad[0]].tolist(), want[bad[0]].tolist())


# Of a number formed in 64 bits by some ten operations, 2^-52 each at most and 2^-48 in all, and rounded once: half a step, and
# where it moves across the middle of one as much more.
ONE_ROUNDING, SMALLEST = 2.0 ** -24 + 2.0 ** -44, 0.51 * 2.0 ** -149


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (9, 63, 5), (300, 256, 8), (5000, 40, 4), (3000, 256, 8), (2500, 500, 16), (2500, 1000, 3)])
@pytest.mark.parametrize("size", [2.0, 30.0, 400.0])
def test_weights_are_rounded_once(T, E, k, score, renormalize, size):
    say("weights", T, E, k, score, renormalize, size)
    g = torch.Generator().manual_seed(E + k)
    logits = torch.randn(T, E, generator=g) * size
    logits[::3] -= 2 * size  # scores that vanish
    logits[::4][torch.rand(len(logits[::4]), E, generator=g) < 0.3] = -INF
    rule = N.make_gate(score, renormalize=renormalize, scale=1.7)
    for bias in (None, torch.randn(E, generator=g) * 0.1):
        idx, w = gate(logits, bias, k, rule)
        want = weights(logits, torch.where(idx >= 0, idx, E), score, renormalize, 1.7)
        off = (w.double() - want).abs() - ONE_ROUNDING * want - SMALLEST
        assert (off <= 0).all(), "%d, one %s" % ((off > 0).sum(), (w[off > 0][0].item(), want[off > 0][0].item()))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (9, 63, 5), (300, 256, 8), (3000, 257, 8), (2500, 600, 16), (50, 1000, 3)])
@pytest.mark.parametrize("size", [2.0, 30.0, 300.0])
def test_gradients_are_rounded_once(T, E, k, score, renormalize, size):
    """An expert may be there twice; entries of experts that are off or out of range take no part."""
    say("gradients", T, E, k, score, renormalize, size)
    g = torch.Generator().manual_seed(E + k)
    logits = torch.randn(T, E, generator=g) * size
    logits[::3] -= 2 * size
    logits[::4][torch.rand(len(logits[::4]), E, generator=g) < 0.3] = -INF
    idx = torch.randint(-1, E + 1, (T, k), generator=g, dtype=torch.int32)
    dw = torch.randn(T, k, generator=g)
    got = torch.full((T, E), 77.0, device=DEV)
    N.moe_gate_backward(shape(T, E, k), N.make_gate(score, renormalize=renormalize, scale=1.7), logits.to(DEV), idx.to(DEV), dw.to(DEV), got)
    l, e = logits.double(), idx.long().clamp(0, E - 1)
    v = l.gather(1, e)
    here = (idx >= 0) & (idx < E) & (v > -INF)
    d = torch.where(here, dw.double(), 0.0)
    at = torch.where(here, e, E)
    w = weights(logits, at, score, renormalize, 1.0)  # r, or the scores
    sums = lambda t: torch.zeros(T, E + 1, dtype=torch.float64).scatter_add_(1, at, t)[:, :E]  # noqa: E731
    if renormalize or score == "softmax":
        mean, most = (w * d).sum(1, keepdim=True), (w * d.abs()).sum(1, keepdim=True)
    else:
        mean = most = torch.zeros(T, 1, dtype=torch.float64)
    if score == "softmax" and not renormalize:
        s = weights(logits, torch.arange(E).expand(T, E), score, False, 1.0)
        s = torch.where(l > -INF, s, 0.0)
        want, added = 1.7 * s * (sums(d) - mean), 1.7 * s * (sums(d.abs()) + most)
    else:
        f = 1.7 * torch.where(here, w * (torch.sigmoid(-v) if score == "sigmoid" else 1.0), 0.0)
        want, added = sums(f * (d - mean)), sums(f * (d.abs() + most))
    # of what is added and may cancel 2^-44 as well
    off = (got.cpu().double() - want).abs() - ONE_ROUNDING * want.abs() - 2.0 ** -44 * added - SMALLEST
    assert (off <= 0).all(), "%d, one %s" % ((off > 0).sum(), (got.cpu()[off > 0][0].item(), want[off > 0][0].item()))


@pytest.mark.parametrize("T", [500, 2300])
@pytest.mark.parametrize("E,k", [(24, 3), (64, 6), (256, 8), (300, 16), (768, 6)])
def test_many_equal_choices(T, E, k):
    """Logits of few values and a bias of one or two: equal choices at the border, above it, and at several values above it."""
    g = torch.Generator().manual_seed(E + T)
    for step, biases in ((0.25, (0.0, 0.0)), (0.5, (0.0, 0.125)), (0.015625, (0.0, 0.0))):
        logits = (torch.randn(T, E, generator=g) / step).round() * step
        bias = torch.tensor(biases)[torch.randint(0, 2, (E,), generator=g)]
        idx, _ = gate(logits, bias, k, N.make_gate("sigmoid"))
        assert torch.equal(idx, by_choices(logits, bias, k)), (step, biases)
