"""Routing of logits and biases that hold the type's lowest value, in batches in which every warp takes many tokens.

Such values are ordinary keys: lower than all others, above those of closed experts (-inf), and no sum or bound that is
made of them may lose that.  Ids are compared for equality with a 64-bit form.  A key of a masked expert is that value
plus a score, which 64 bits would round away: the plain form has -64 in the value's place, an order of the same numbers
(all other keys lie within -8 .. 8) to 2^-47; the logits are whole sixteenths there, so that scores are equal or differ by
more than 2^-24 of themselves, what two floats keep of such a key.  Weights: 2^-18 relative, the means of the scores one bit more.
"""
from __future__ import annotations

import pytest
import torch

from counting_sort_bucketization_gb300 import binding, build

pytestmark = pytest.mark.gpu

DEV = "cuda"
FP32, BF16 = torch.float32, torch.bfloat16
LOWEST = torch.finfo(FP32).min


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.load_library()


def plain(l, b, K, score, G, kept, group_sum):
    """Ids, normalised weights and the means of the scores' shares (of their logarithms: they may be below 64 bits)."""
    N, E = l.shape
    x = l.double()
    shift = torch.zeros(E, dtype=torch.float64, device=DEV) if b is None else torch.where(b.abs() == -LOWEST, 64.0 * b.sign(), b).double()
    open_ = (x > float("-inf")) & (shift > float("-inf"))
    s = torch.sigmoid(x) if score == "sigmoid" else torch.nan_to_num(torch.softmax(x, 1))
    key = torch.where(open_, s + shift, float("-inf"))
    order = torch.where(open_, x, float("-inf")) if b is None else key
    if kept < G:
        best = torch.sort(key.view(N, G, -1), dim=2, descending=True).values[:, :, :group_sum]
        total = torch.where(best > float("-inf"), best, 0.0).sum(2)
        total = torch.where(best[:, :, 0] > float("-inf"), total, float("-inf"))
        top = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :kept]
        keep = torch.zeros((N, G), dtype=torch.bool, device=DEV).scatter_(1, top, True)
        order = torch.where(keep.repeat_interleave(E // G, 1), order, float("-inf"))
    order = torch.nn.functional.pad(order, (0, max(0, K - E)), value=float("-inf"))
    top = torch.sort(order, dim=1, descending=True, stable=True)
    ids = torch.where(top.values[:, :K] > float("-inf"), top.indices[:, :K], -1)
    log = torch.nn.functional.logsigmoid(x) if score == "sigmoid" else x
    w = torch.nan_to_num(torch.softmax(torch.where(ids >= 0, log.gather(1, ids.clamp(min=0)), float("-inf")), 1))
    routed = open_.any(1, keepdim=True)
    mean = (torch.nan_to_num(torch.softmax(log, 1)) * routed).sum(0) / routed.sum().clamp(min=1)
    return ids, 2.5 * w, mean, int(routed.sum())


def check(l, b, K, score, G=1, kept=1, group_sum=1, want=None):
    N, E = l.shape
    gate = binding.Gate(binding.LayoutDesc(N, K, E, 1, 1),
                        binding.GateConfig(score, True, 2.5, 0.02, bias_on="score", num_groups=G, topk_groups=kept, group_sum=group_sum))
    ids, w, mean, routed = plain(l, b, K, score, G, kept, group_sum) if want is None else want
    wide = torch.full((N + 1, E + 5), float("nan"), dtype=l.dtype, device=DEV)     # rows apart, with NaN between
    wide[:N, :E] = l
    for rows in (l, wide[:N, :E]):
        gate.forward(rows, bias=b)
        assert torch.equal(gate.topk_idx, ids)
        assert torch.equal(gate.expert_count.long(), torch.bincount(ids[ids >= 0], minlength=E))
        assert int(gate.routed_tokens) == routed and gate.error() == 0
        assert torch.all((gate.prob_mean.double() - mean).abs() <= 2.0 ** -17 * mean + 1e-30)
        assert torch.all((gate.weights.double() - w).abs() <= 2.0 ** -18 * w + 1e-30)
    return gate


def draw(N, E, seed, dtype=FP32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    l = (torch.randn((N, E), generator=g, device=DEV) * 1.5).to(dtype)
    return l, torch.randn(E, generator=g, device=DEV) * 0.05, lambda p, *s: torch.rand(s, generator=g, device=DEV) < p


EXPERTS = [(8, 2, 1, 1), (16, 4, 1, 1), (31, 8, 1, 1), (32, 8, 1, 1), (33, 6, 1, 1), (16, 2, 8, 2), (64, 6, 8, 2), (96, 8, 12, 1),
           (256, 8, 8, 4)]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [FP32, BF16])
@pytest.mark.parametrize("E,K,G,kept", EXPERTS)
def test_logits_of_the_lowest_value(E, K, G, kept, dtype, score):
    """Padding rows of nothing else, single experts masked by it, closed experts and empty rows among ordinary ones."""
    N = 20000
    l, b, some = draw(N, E, E + K, dtype)
    low = torch.finfo(dtype).min
    l = torch.where(some(0.3, N, E), low, l)
    l = torch.where(some(0.1, N, E), float("-inf"), l)
    l = torch.where(some(0.2, N, 1), low, l)
    l = torch.where(some(0.05, N, 1), float("-inf"), l)
    one = torch.where(some(0.1, N, 1) & (torch.arange(E, device=DEV) != 3), low, l)      # one expert beside the lowest values
    check(one, None, K, score, G, kept)
    check(one, b if score == "sigmoid" else b * 0.1, K, score, G, kept)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,K,G,kept", EXPERTS)
def test_biases_of_the_lowest_value(E, K, G, kept, score):
    """Experts masked by their bias, down to fewer than K others; closed ones beside them are never taken."""
    N = 6000
    l, b, some = draw(N, E, 3 * E + K)
    l = torch.where(some(0.1, N, E), float("-inf"), torch.round(l * 16) / 16)
    b = b if score == "sigmoid" else b * 0.1
    for open_ in (E - 1, E // 2, 1, 0):
        masked = torch.where(torch.arange(E, device=DEV) < open_, b, LOWEST)
        masked[E // 3] = float("-inf")
        check(l, masked, K, score, G, kept)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("value", [LOWEST, -LOWEST])
@pytest.mark.parametrize("E,G,kept,K", [(24, 3, 1, 4), (24, 3, 2, 6), (64, 8, 4, 6), (64, 32, 5, 6), (96, 12, 7, 12), (256, 8, 3, 8), (60, 12, 4, 8)])
def test_groups_of_extreme_biases(E, G, kept, K, value, score):
    """Two such keys add to the group's score without an overflow: a masked group is the last that stays, above closed
    ones, and never before another; one of the largest value is the first.  Also where every choice of groups is left
    open (all biases and scores equal but for the masked groups')."""
    per = E // G
    l, b, some = draw(6000, E, 5 * E + G)
    l = torch.round(l * 16) / 16 + 2.0 ** -6          # no two whose sigmoids add to one
    b = b if score == "sigmoid" else b * 0.1
    g = torch.arange(E, device=DEV) // per
    for some_groups in ([1], [0, 2], list(range(1, G)), list(range(G))):
        b2 = torch.where(torch.isin(g, torch.tensor(some_groups, device=DEV)), value, b)
        check(l, b2, K, score, G, kept, 2)
        b2[0] = b2[E // 2] = float("-inf")
        check(l, b2, K, score, G, kept, 2)
        b2 = torch.where(torch.isin(g, torch.tensor(some_groups, device=DEV)), value, 0.25 * (torch.arange(E, device=DEV) % per % 2))
        check(torch.zeros_like(l), b2, K, score, G, kept, 2)
