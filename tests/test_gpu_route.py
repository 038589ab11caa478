"""Routing by score + bias and by groups of experts against a plain 64-bit implementation.

The choice of experts is compared for equality: keys are numbers in 64 bits, and no case here has two that differ
by less than 2^-45 without being equal.  Weights, means and loss as the gate's: 64 * 2^-24 = 2^-18 relative for a score
or a weight, one bit more for a sum over tokens, two for the loss.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from counting_sort_bucketization_gb300 import binding, build

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.load_library()


def plain(l32, bias, K, score, G, topk_groups, group_sum, normalize=True, scale=2.5, coef=0.02, by_logit=False):
    """``by_logit``: scores whose 64-bit values may be equal where the logits are not are ordered by the logits."""
    N, E = l32.shape
    l = l32.astype(np.float64)
    with np.errstate(all="ignore"):
        if score == "softmax":
            m = l.max(1, keepdims=True)
            s = np.exp(l - np.where(np.isfinite(m), m, 0.0))
            s = s / np.maximum(s.sum(1, keepdims=True), 1e-300)
        else:
            s = 1 / (1 + np.exp(-l))
    key = s + (0.0 if bias is None else bias.astype(np.float64))
    key[np.isneginf(l)] = -np.inf
    idx = np.full((N, K), -1, np.int64)
    routed = (key > -np.inf).any(1)
    for t in range(N):
        rank = (lambda e: (-l[t, e], e)) if by_logit else (lambda e: (-key[t, e], e))
        groups = []
        for g in range(G):
            own = sorted((k for k in key[t, g * E // G:(g + 1) * E // G] if k > -np.inf), reverse=True)[:group_sum]
            if own:
                groups.append((-sum(own), g))
        kept = {g for _, g in sorted(groups)[:topk_groups]} if topk_groups < G else set(range(G))
        picks = sorted((e for e in range(E) if key[t, e] > -np.inf and e // (E // G) in kept), key=rank)[:K]
        idx[t, :len(picks)] = picks
    s[~routed] = 0
    total = np.maximum(s.sum(1, keepdims=True), 1e-300)
    got = np.where(idx >= 0, np.take_along_axis(s, np.maximum(idx, 0), 1), 0.0)
    D = np.maximum(got.sum(1, keepdims=True), 1e-300) if normalize else np.ones((N, 1))
    T = int(routed.sum())
    count = np.bincount(idx[idx >= 0], minlength=E)
    mean = (s / total).sum(0) / max(T, 1)
    f = count / (K * max(T, 1))
    return dict(idx=idx, weights=scale * got / D, count=count, mean=mean, loss=coef * E * float((f * mean).sum()), T=T)


def route(l, b, K, score, G=1, topk_groups=1, group_sum=1, normalize=True, stride=None):
    N, E = l.shape
    cfg = binding.GateConfig(score, normalize, 2.5, 0.02, bias_on="score", num_groups=G, topk_groups=topk_groups,
                             group_sum=group_sum)
    gate = binding.Gate(binding.LayoutDesc(N, K, E, 1, 1), cfg)
    ld = l.to(DEV)
    if stride:
        wide = torch.full((N, stride), float("nan"), dtype=l.dtype, device=DEV)
        wide[:, :E] = ld
        ld = wide[:, :E]
    return gate.forward(ld, bias=None if b is None else b.to(DEV))


def check(gate, r):
    np.testing.assert_array_equal(gate.topk_idx.cpu().numpy(), r["idx"])
    np.testing.assert_array_equal(gate.expert_count.cpu().numpy(), r["count"])
    assert int(gate.routed_tokens) == r["T"]
    w = gate.weights.double().cpu().numpy()
    assert np.all(np.abs(w - r["weights"]) <= 2.0 ** -18 * np.abs(r["weights"]) + 1e-30)
    m = gate.prob_mean.double().cpu().numpy()
    assert np.all(np.abs(m - r["mean"]) <= 2.0 ** -17 * r["mean"] + 1e-30)
    assert abs(float(gate.loss) - r["loss"]) <= 2.0 ** -16 * abs(r["loss"])


def draw(N, E, seed, dtype=torch.float32, closed=0.0, empty=0.0, bias=0.05, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn((N, E), generator=g) * spread
    if closed:
        l[torch.rand((N, E), generator=g) < closed] = float("-inf")
    if empty:
        l[torch.rand(N, generator=g) < empty] = float("-inf")
    b = torch.randn(E, generator=g) * bias if bias else None
    return l.to(dtype), b


CASES = [
    # N, E, K, G, topk_groups, group_sum, dtype, score, normalize, bias, closed, empty
    (1, 1, 1, 1, 1, 1, torch.float32, "sigmoid", True, 0.1, 0, 0),
    (2, 8, 3, 8, 2, 2, torch.float32, "sigmoid", True, 0.1, 0, 0),          # groups of one expert
    (64, 256, 8, 8, 4, 2, torch.float32, "sigmoid", True, 0.05, 0, 0),
    (300, 256, 8, 8, 4, 2, torch.float32, "softmax", True, 0.001, 0, 0),
    (257, 384, 8, 16, 4, 2, torch.float32, "sigmoid", True, 0.05, 0, 0.05),
    (301, 40, 3, 4, 2, 1, torch.bfloat16, "softmax", True, 0.01, 0.2, 0.05),
    (130, 60, 12, 12, 5, 2, torch.bfloat16, "sigmoid", False, 0.2, 0.5, 0.1),   # groups with few open experts
    (95, 64, 6, 32, 7, 2, torch.bfloat16, "softmax", False, 0.0, 0.5, 0.1),
    (95, 64, 6, 2, 1, 1, torch.bfloat16, "sigmoid", True, 0.0, 0.1, 0.1),
    (77, 100, 1, 5, 1, 2, torch.float32, "sigmoid", True, 0.3, 0, 0),
    (50, 512, 8, 8, 3, 2, torch.float32, "sigmoid", True, 0.05, 0, 0),
    (40, 1000, 16, 20, 10, 2, torch.bfloat16, "sigmoid", True, 0.05, 0.1, 0),
    (41, 1024, 32, 32, 8, 1, torch.float32, "softmax", True, 0.0005, 0, 0),
    (60, 33, 8, 3, 2, 2, torch.float32, "sigmoid", True, 0.05, 0.3, 0.1),
    (60, 30, 32, 3, 1, 2, torch.float32, "sigmoid", True, 0.05, 0.3, 0.1),  # more slots than experts
    (3000, 48, 4, 1, 1, 1, torch.float32, "sigmoid", True, 0.05, 0, 0),     # a score bias without groups
    (200, 37, 5, 1, 1, 1, torch.bfloat16, "softmax", True, 0.02, 0.1, 0.05),
]


@pytest.mark.parametrize("N,E,K,G,topk_groups,group_sum,dtype,score,normalize,bias,closed,empty", CASES)
def test_forward(N, E, K, G, topk_groups, group_sum, dtype, score, normalize, bias, closed, empty):
    l, b = draw(N, E, 100 + N + E, dtype, closed, empty, bias)
    r = plain(l.float().numpy(), None if b is None else b.numpy(), K, score, G, topk_groups, group_sum, normalize)
    for stride in (None, E + 3):
        gate = route(l, b, K, score, G, topk_groups, group_sum, normalize, stride)
        assert gate.error() == 0
        check(gate, r)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,topk_groups", [(64, 1, 1), (64, 4, 2), (256, 8, 3), (520, 8, 4)])
def test_keys_that_32_bits_cannot_order(score, E, G, topk_groups):
    """Biases that make every key of a row the same to about 2^-24: their order is that of the 64-bit sums."""
    g = torch.Generator().manual_seed(E + G)
    base = torch.randn(E, generator=g) * 1.5
    s = torch.sigmoid(base.double()) if score == "sigmoid" else torch.softmax(base.double(), 0)
    b = (0.75 - s).float()
    step = 2.0 ** -22 * torch.randint(-8, 9, (70, E), generator=g)
    l = base + step * base.abs()
    r = plain(l.numpy(), b.numpy(), 6, score, G, topk_groups, 2)
    gate = route(l, b, 6, score, G, topk_groups, 2)
    assert gate.error() == 0
    check(gate, r)


@pytest.mark.parametrize("bias", ["none", "zeros", "same", "few"])
@pytest.mark.parametrize("value", [0.0, 3.5, -200.0, torch.finfo(torch.float32).min])
@pytest.mark.parametrize("G,topk_groups", [(1, 1), (6, 3)])
def test_equal_logits(bias, value, G, topk_groups):
    """All logits the same (a router of zeros, rows masked by the type's lowest value): ties go to the lower id."""
    N, E, K = 9, 96, 7
    l = torch.full((N, E), value)
    l[1:, 5], l[2:, 77] = value + 1.0, value + 2.0
    b = {"none": None, "zeros": torch.zeros(E), "same": torch.full((E,), 0.25), "few": torch.arange(E) % 3 * 0.5}[bias]
    r = plain(l.numpy(), None if b is None else b.numpy(), K, "softmax", G, topk_groups, 2)
    gate = route(l, b, K, "softmax", G, topk_groups, 2)
    assert gate.error() == 0
    check(gate, r)


def test_saturated_sigmoids_without_a_bias_go_by_logit():
    """Scores that 64 bits cannot tell apart either: without a bias the larger logit comes first."""
    l = torch.arange(64, dtype=torch.float32).repeat(5, 1) + 40.0
    for E, G, kept in ((64, 1, 1), (64, 4, 2)):
        gate = route(l, None, 8, "sigmoid", G, kept, 1)
        r = plain(l.numpy(), None, 8, "sigmoid", G, kept, 1, by_logit=True)
        if G == 1:
            np.testing.assert_array_equal(gate.topk_idx.cpu().numpy(), r["idx"])
        else:
            assert gate.topk_idx[0].tolist() == list(range(63, 55, -1))
        assert gate.error() == 0


def test_tiny_sigmoids():
    """Rows whose scores all but vanish: without a bias their order and shares are kept, with one it decides."""
    l, b = draw(50, 64, 5, spread=4.0)
    l = l - 60.0
    check(route(l, None, 6, "sigmoid", 4, 2, 2), plain(l.numpy(), None, 6, "sigmoid", 4, 2, 2))
    check(route(l, b, 6, "sigmoid", 4, 2, 2), plain(l.numpy(), b.numpy(), 6, "sigmoid", 4, 2, 2))


def test_rows_that_cannot_be_routed():
    """NaN and +inf are recorded, rows without an open expert are not; both route nowhere."""
    l, b = draw(8, 32, 6)
    l[1, 3], l[2, 4], l[3], l[4, 9] = float("nan"), float("inf"), float("-inf"), -float("nan")
    r = plain(torch.where(torch.isfinite(l).all(1, keepdim=True), l, float("-inf")).numpy(), b.numpy(), 4, "sigmoid", 4, 2, 2)
    gate = route(l, b, 4, "sigmoid", 4, 2, 2)
    assert gate.error() == 1 and gate.error() == 0
    check(gate, r)
    gate = route(l[:1], torch.where(torch.arange(32) == 7, float("nan"), b), 4, "sigmoid", 4, 2, 2)
    assert gate.error() == 1 and torch.all(gate.topk_idx == -1) and int(gate.routed_tokens) == 0
    # the same where every group ties, so that the groups alone would leave the choice open
    for value in (float("nan"), float("inf")):
        gate = route(torch.zeros((40, 32)), torch.where(torch.arange(32) == 7, value, torch.arange(32) % 8 * 0.1), 4, "sigmoid", 4, 2, 2)
        assert gate.error() == 1 and torch.all(gate.topk_idx == -1) and torch.all(gate.weights == 0)
        assert int(gate.routed_tokens) == 0 and int(gate.expert_count.sum()) == 0


def test_experts_closed_by_their_bias():
    l, b = draw(40, 48, 7)
    b[:16], b[20] = float("-inf"), float("-inf")
    r = plain(l.numpy(), b.numpy(), 8, "sigmoid", 3, 2, 2)
    check(route(l, b, 8, "sigmoid", 3, 2, 2), r)
    assert torch.all(route(l, torch.full((48,), float("-inf")), 8, "sigmoid", 3, 2, 2).topk_idx == -1)


@pytest.mark.parametrize("N", [0, 1, 5000])
def test_sizes_and_repeats(N):
    l, b = draw(N, 72, 8, bias=0.05)
    gate = route(l, b, 4, "sigmoid", 6, 2, 2)
    first = [t.clone() for t in (gate.topk_idx, gate.weights, gate.expert_count, gate.prob_mean, gate.loss)]
    r = plain(l.numpy(), b.numpy(), 4, "sigmoid", 6, 2, 2)
    check(gate, r)
    gate.forward(l.to(DEV), bias=b.to(DEV))
    for a, c in zip(first, (gate.topk_idx, gate.weights, gate.expert_count, gate.prob_mean, gate.loss)):
        assert torch.equal(a, c)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_autograd_and_differences(score):
    """The gate's gradient on this choice: the formula by autograd in 64 bits, and differences of the forward pass.

    Autograd: 2^-14 of the largest gradient.  Differences: a step of 2^-7 in one logit errs by the third derivative,
    2^-14 / 6 of values of order one, and by 2^-18 * 2.5 of two forward results over 2^-6: 2^-10 of the row's sum."""
    N, E, K = 30, 24, 4
    l, b = draw(N, E, 9)
    gate = route(l, b, K, score, 4, 2, 2)
    dw = torch.randn((N, K), generator=torch.Generator().manual_seed(2)).to(DEV)
    ld = l.to(DEV)
    dl = gate.backward(ld, torch.empty_like(ld), dw, torch.ones(1, device=DEV))
    leaf = ld.double().requires_grad_()
    s = torch.sigmoid(leaf) if score == "sigmoid" else torch.softmax(leaf, 1)
    wk = s.gather(1, gate.topk_idx)
    f = gate.expert_count.double() / (K * N)
    loss = 0.02 * E * (f * (s / s.sum(1, keepdim=True)).mean(0)).sum()
    ((2.5 * wk / wk.sum(1, keepdim=True) * dw).sum() + loss).backward()
    assert float((dl.double() - leaf.grad).abs().max()) <= 2.0 ** -14 * float(leaf.grad.abs().max())
    ids = gate.topk_idx.clone()
    for e in ids[:, 0].unique().tolist()[:4]:
        side = []
        for step in (2.0 ** -7, -2.0 ** -7):
            moved = ld.clone()
            moved[:, e] += step
            g2 = route(moved.cpu(), b, K, score, 4, 2, 2)
            side.append((torch.equal(g2.topk_idx, ids), (g2.weights * dw).sum(1), g2.topk_idx.clone()))
        same = (side[0][2] == ids).all(1) & (side[1][2] == ids).all(1)     # rows whose choice stays
        diff = (side[0][1] - side[1][1]) * 2.0 ** 6
        own = torch.zeros_like(dw)
        only = gate.backward(ld, torch.empty_like(ld), dw, None)
        assert int(same.sum()) > 10
        assert torch.all(((diff - only[:, e]).abs() <= 2.0 ** -10 * (2.5 * dw.abs().sum(1) + 1))[same])


def test_graph_replay_on_another_stream():
    l, b = draw(100, 64, 10)
    gate = route(l, b, 4, "sigmoid", 4, 2, 2)
    ld, bd = l.to(DEV), b.to(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gate.forward(ld, bias=bd)
    l2, _ = draw(100, 64, 11)
    ld.copy_(l2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph.replay()
    s.synchronize()
    check(gate, plain(l2.numpy(), b.numpy(), 4, "sigmoid", 4, 2, 2))
    assert gate.error() == 0
