"""Routing of rows whose groups of experts tie: padding rows of equal logits, with biases that are the same or whole steps.

Groups that tie exactly go by their ids, without a look at keys of more than 32 bits: a batch of such rows takes about
twice an ordinary one's time (their keys are all candidates, more than a list holds: K + 1 passes over a lane's columns,
as many instructions as the rest of a token), one of open tokens alone five times; three times is the limit here.
Groups that only look equal in 32 bits are told apart.

Ids against 64-bit torch.  Keys are told apart to about 2^-46 of themselves: a token of which two deciding keys lie closer
than 2^-45 without being equal is not compared, nor one whose border groups' sums lie so close and are sums of different
keys: these may be equal as numbers, which no number of bits shows (sigmoid(x) + sigmoid(-x) is 1 for every x, and
(s + b) + s' is s + (s' + b); 64 bits round each in its own way).
"""
from __future__ import annotations

import pytest
import torch

from counting_sort_bucketization_gb300 import binding, build

pytestmark = pytest.mark.gpu

DEV = "cuda"
SHAPES = [(384, 8, 16, 4, 2), (256, 8, 8, 4, 2), (256, 8, 8, 3, 1), (160, 6, 8, 3, 2), (64, 4, 32, 5, 2), (60, 6, 12, 5, 2), (33, 8, 3, 2, 2),
          (1000, 8, 20, 6, 2)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.load_library()


def new_gate(N, E, K, score, G, kept, group_sum):
    return binding.Gate(binding.LayoutDesc(N, K, E, 1, 1),
                        binding.GateConfig(score, True, 2.5, 0.02, bias_on="score", num_groups=G, topk_groups=kept, group_sum=group_sum))


def check(l, b, K, score, G, kept, group_sum, at_most):
    """``at_most``: the share of tokens that may be too close to compare."""
    N, E = l.shape
    gate = new_gate(N, E, K, score, G, kept, group_sum).forward(l, bias=b)
    x = l.double()
    s = torch.sigmoid(x) if score == "sigmoid" else torch.nan_to_num(torch.softmax(x, 1))
    key = torch.where(x > float("-inf"), s + (0.0 if b is None else b.double()), float("-inf"))
    best = torch.sort(key.view(N, G, -1), dim=2, descending=True).values[:, :, :group_sum]
    total = torch.where(best > float("-inf"), best, 0.0).sum(2)
    total = torch.where(best[:, :, 0] > float("-inf"), total, float("-inf"))
    top = torch.sort(total, dim=1, descending=True, stable=True)
    border = ((total - top.values[:, kept - 1:kept]).abs() < 2.0 ** -45).unsqueeze(2)
    terms = [torch.where(border, best, end * float("inf")) for end in (1, -1)]
    undecided = (terms[0].amin(1) != terms[1].amax(1)).any(1) & (border.sum((1, 2)) > 1)
    near = lambda gap: (gap > 0) & (gap < 2.0 ** -45)
    keep = torch.zeros((N, G), dtype=torch.bool, device=DEV).scatter_(1, top.indices[:, :kept], True)
    order = torch.where(keep.repeat_interleave(E // G, 1) & (x > float("-inf")), x if b is None else key, float("-inf"))
    top = torch.sort(order, dim=1, descending=True, stable=True)
    if b is not None:
        undecided |= near(top.values[:, :K] - top.values[:, 1:K + 1]).any(1)
    ids = torch.where(top.values[:, :K] > float("-inf"), top.indices[:, :K], -1)
    assert int(undecided.sum()) <= at_most * N
    assert torch.equal(gate.topk_idx[~undecided], ids[~undecided])
    assert gate.error() == 0


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,K,G,kept,group_sum", SHAPES)
def test_equal_rows(E, K, G, kept, group_sum, score):
    N = 12000
    g = torch.Generator(device=DEV).manual_seed(E + G)
    l = torch.randn((N, E), generator=g, device=DEV) * 1.5
    rows = torch.rand((N, 1), generator=g, device=DEV)
    l = torch.where(rows < 0.3, 0.0, l)                                     # zeros
    l = torch.where((rows >= 0.3) & (rows < 0.5), torch.round(l), l)        # few values: groups of the same two largest
    l = torch.where((rows >= 0.5) & (rows < 0.6) & (torch.rand((N, E), generator=g, device=DEV) < 0.6), float("-inf"), torch.where(rows < 0.6, torch.round(l), l))
    few = torch.randint(-1, 2, (E,), generator=g, device=DEV) * 2.0 ** -10
    for b in (None, torch.zeros(E, device=DEV), torch.full((E,), 0.25, device=DEV), few, few * 64):
        check(l, b, K, score, G, kept, group_sum, 0.1)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,K,G,kept,group_sum", SHAPES)
def test_groups_equal_in_32_bits_only(E, K, G, kept, group_sum, score):
    """Keys within 2^-22 of each other, of other logits and biases; without a bias, logits a few units apart."""
    N = 4000
    g = torch.Generator(device=DEV).manual_seed(E)
    base = torch.randn(E, generator=g, device=DEV) * 1.5
    s = torch.sigmoid(base.double()) if score == "sigmoid" else torch.softmax(base.double(), 0)
    l = base + 2.0 ** -22 * torch.randint(-8, 9, (N, E), generator=g, device=DEV) * base.abs()
    check(l, (0.75 - s).float(), K, score, G, kept, group_sum, 0.05)
    l = 1.0 + 2.0 ** -23 * torch.randint(0, 3, (N, E), generator=g, device=DEV)
    check(l, None, K, score, G, kept, group_sum, 0.05)
    check(l, torch.full((E,), 0.25, device=DEV), K, score, G, kept, group_sum, 0.05)


@pytest.mark.parametrize("biased", [False, True])
def test_padding_rows_are_not_left_open(biased):
    N, E = 131072, 384
    g = torch.Generator(device=DEV).manual_seed(1)
    l = torch.randn((N, E), generator=g, device=DEV) * 1.5
    gate = new_gate(N, E, 8, "sigmoid", 16, 4, 2)
    b = torch.where(torch.arange(E, device=DEV) % 3 == 0, 2.0 ** -10, 0.0) if biased else None     # each group has the same two largest
    best = []
    for rows in (l, torch.zeros_like(l)):
        times = []
        for _ in range(8):
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            gate.forward(rows, bias=b)
            end.record()
            torch.cuda.synchronize()
            times.append(start.elapsed_time(end))
        best.append(min(times))
    assert torch.equal(gate.topk_idx[:, 0], torch.zeros(N, dtype=torch.int64, device=DEV))
    assert best[1] < 3 * best[0]
