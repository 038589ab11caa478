"""Routing of batches in which every warp takes many tokens, against 64-bit torch on the device.

What a warp learns from one token (where the candidates' bound lies) must not show in another's result, and choices that
32 bits leave open are settled after the loop, however many there are.  Ids are compared for equality; keys that
differ in 64 bits by less than 2^-45 without being equal do not occur (checked).  Weights: 2^-18 relative.
"""
from __future__ import annotations

import pytest
import torch

from counting_sort_bucketization_gb300 import binding, build

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.load_library()


def plain(l, b, K, score, G, kept, group_sum):
    """Ids by the 64-bit keys (by the logits where there is no bias), and the normalised weights."""
    N, E = l.shape
    x = l.double()
    open_ = l > float("-inf")
    s = torch.sigmoid(x) if score == "sigmoid" else torch.nan_to_num(torch.softmax(x, 1))
    key = torch.where(open_, s + (0.0 if b is None else b.double()), float("-inf"))
    order = torch.where(open_, x, float("-inf")) if b is None else key
    if kept < G:
        best = torch.sort(key.view(N, G, -1), dim=2, descending=True).values[:, :, :group_sum]
        total = torch.where(best > float("-inf"), best, 0.0).sum(2)
        total = torch.where(best[:, :, 0] > float("-inf"), total, float("-inf"))
        top = torch.sort(total, dim=1, descending=True, stable=True)
        border = top.values[:, kept - 1] - top.values[:, kept]
        assert not torch.any((border > 0) & (border < 2.0 ** -45))
        keep = torch.zeros((N, G), dtype=torch.bool, device=DEV).scatter_(1, top.indices[:, :kept], True)
        order = torch.where(keep.repeat_interleave(E // G, 1), order, float("-inf"))
    top = torch.sort(order, dim=1, descending=True, stable=True)
    gaps = top.values[:, :K] - top.values[:, 1:K + 1]
    assert b is None or not torch.any((gaps > 0) & (gaps < 2.0 ** -45))
    picked = top.values[:, :K] > float("-inf")
    ids = torch.where(picked, top.indices[:, :K], -1)
    w = torch.where(picked, s.gather(1, top.indices[:, :K]), 0.0)
    return ids, 2.5 * w / w.sum(1, keepdim=True).clamp(min=1e-300)


def check(l, b, K, score, G=1, kept=1, group_sum=1):
    N, E = l.shape
    gate = binding.Gate(binding.LayoutDesc(N, K, E, 1, 1),
                        binding.GateConfig(score, True, 2.5, 0.02, bias_on="score", num_groups=G, topk_groups=kept, group_sum=group_sum))
    gate.forward(l, bias=b)
    ids, w = plain(l, b, K, score, G, kept, group_sum)
    assert torch.equal(gate.topk_idx, ids)
    assert torch.all((gate.weights.double() - w).abs() <= 2.0 ** -18 * w + 1e-30)
    assert torch.equal(gate.expert_count.long(), torch.bincount(ids[ids >= 0], minlength=E))
    assert int(gate.routed_tokens) == int((ids[:, 0] >= 0).sum()) and gate.error() == 0
    first = [t.clone() for t in (gate.topk_idx, gate.weights, gate.prob_mean, gate.loss)]
    gate.forward(l, bias=b)
    for a, c in zip(first, (gate.topk_idx, gate.weights, gate.prob_mean, gate.loss)):
        assert torch.equal(a, c)


def draw(N, E, seed, dtype=torch.float32, bias=0.05, spread=1.5, closed=0.0, empty=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    l = torch.randn((N, E), generator=g, device=DEV) * spread
    if closed:
        l = torch.where(torch.rand((N, E), generator=g, device=DEV) < closed, float("-inf"), l)
    if empty:
        l = torch.where(torch.rand((N, 1), generator=g, device=DEV) < empty, float("-inf"), l)
    return l.to(dtype), (torch.randn(E, generator=g, device=DEV) * bias if bias else None)


@pytest.mark.parametrize("N,E,K,G,kept,group_sum,dtype,score,bias,closed,empty", [
    (40000, 256, 8, 8, 4, 2, torch.float32, "sigmoid", 0.05, 0.0, 0.0),
    (30000, 384, 8, 16, 4, 2, torch.float32, "softmax", 0.0005, 0.0, 0.01),
    (50000, 40, 3, 4, 2, 1, torch.bfloat16, "softmax", 0.005, 0.1, 0.02),
    (25000, 160, 6, 8, 3, 2, torch.float32, "sigmoid", 0.05, 0.0, 0.0),      # groups of 20: not of whole lanes
    (25000, 96, 6, 12, 5, 2, torch.bfloat16, "sigmoid", 0.05, 0.3, 0.0),
    (20000, 33, 8, 1, 1, 1, torch.float32, "sigmoid", 0.05, 0.2, 0.05),      # rows that start off a vector's boundary
    (20000, 64, 12, 1, 1, 1, torch.bfloat16, "softmax", 0.0, 0.0, 0.0),      # many equal logits
    (12000, 1000, 16, 20, 6, 2, torch.bfloat16, "sigmoid", 0.05, 0.0, 0.0),
    (12000, 512, 32, 4, 1, 1, torch.float32, "sigmoid", 0.05, 0.0, 0.0),
    (20000, 128, 1, 1, 1, 1, torch.float32, "sigmoid", 0.05, 0.0, 0.0),
])
def test_batches(N, E, K, G, kept, group_sum, dtype, score, bias, closed, empty):
    l, b = draw(N, E, N + E, dtype, bias, closed=closed, empty=empty)
    check(l, b, K, score, G, kept, group_sum)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,kept", [(64, 1, 1), (64, 4, 2), (240, 12, 5)])
def test_rows_of_every_scale(score, E, G, kept):
    """Rows whose keys lie elsewhere than the last token's: spreads from 2^-8 to 2^4, and shifts."""
    l, b = draw(20000, E, 3)
    g = torch.Generator(device=DEV).manual_seed(4)
    l = l * torch.exp2(torch.randint(-8, 4, (20000, 1), generator=g, device=DEV).float()) + torch.randint(-6, 7, (20000, 1), generator=g, device=DEV)
    check(l, b if score == "sigmoid" else b * 0.1, 6, score, G, kept, 2)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,kept", [(64, 1, 1), (64, 4, 2)])
def test_every_choice_left_open(score, E, G, kept):
    """Biases that bring all keys within 2^-22 of each other: many open tokens a warp, in both kinds."""
    g = torch.Generator(device=DEV).manual_seed(5)
    base = torch.randn(E, generator=g, device=DEV) * 1.5
    s = torch.sigmoid(base.double()) if score == "sigmoid" else torch.softmax(base.double(), 0)
    l = base + 2.0 ** -22 * torch.randint(-8, 9, (15000, E), generator=g, device=DEV) * base.abs()
    check(l, (0.75 - s).float(), 6, score, G, kept, 2)


@pytest.mark.parametrize("bias", [None, 0.0, 0.5])
def test_a_router_of_zeros(bias):
    l = torch.zeros((20000, 96), device=DEV)
    l[::7, 50] = 1.0
    check(l, None if bias is None else torch.full((96,), bias, device=DEV), 8, "sigmoid", 6, 2, 2)
    check(l, torch.arange(96, device=DEV) % 5 * 0.25, 8, "sigmoid", 6, 2, 2)


def test_the_function_gives_what_the_object_gives():
    l, b = draw(3000, 64, 9)
    desc = binding.LayoutDesc(3000, 4, 64, 1, 1)
    cfg = binding.GateConfig("sigmoid", True, 2.5, 0.02, bias_on="score", num_groups=8, topk_groups=3, group_sum=2)
    gate = binding.Gate(desc, cfg).forward(l, bias=b)
    out = [torch.empty_like(t) for t in (gate.topk_idx, gate.weights, gate.expert_count, gate.prob_mean, gate.routed_tokens, gate.loss)]
    ws = binding.new_gate_workspace(desc)
    binding.gate_forward(desc, cfg, l, *out, ws, bias=b)
    for t, want in zip(out, (gate.topk_idx, gate.weights, gate.expert_count, gate.prob_mean, gate.routed_tokens, gate.loss)):
        assert torch.equal(t, want)
    assert binding.get_error(ws) == 0
    dw = torch.randn((3000, 4), device=DEV)
    got = binding.gate_backward(desc, cfg, l, out[0], out[2], out[4], torch.empty_like(l), ws, dweights=dw)
    assert got is None
