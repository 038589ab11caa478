"""The top-k gate and its gradient against a plain 64-bit implementation.

Tolerances.  A score is exp, a sum over E and a division in fp32: expf and the
sum err by a few 2^-24 each, |l - max| <= 32 adds 2^-24 * 32 at most to the
argument.  64 * 2^-24 = 2^-18 relative bounds a score and a weight; a sum over
tokens keeps it, plus one rounding per addition of a lane, 2^-24 each.
Gradients are sums of products of those with cancellation: 2^-16 of the sum of
the magnitudes that enter them.
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


def plain(l32, bias, K, score, normalize, scale, coef):
    """Ids by the 32-bit key; everything else in 64 bits."""
    N, E = l32.shape
    key = (l32 + (bias if bias is not None else np.float32(0))).astype(np.float32)
    idx = np.full((N, K), -1, np.int64)
    for t in range(N):
        order = sorted(range(E), key=lambda e: (-key[t, e], e))[:K]
        picks = [e for e in order if key[t, e] > -np.inf]
        idx[t, : len(picks)] = picks
    routed = idx[:, 0] >= 0
    l = l32.astype(np.float64)
    with np.errstate(all="ignore"):
        if score == "softmax":
            s = np.exp(l - np.where(routed, l.max(1), 0.0)[:, None])
            s = s / np.maximum(s.sum(1, keepdims=True), 1e-300)
        else:
            s = 1 / (1 + np.exp(-l))
    s[~routed] = 0
    total = np.maximum(s.sum(1, keepdims=True), 1e-300)
    got = np.where(idx >= 0, np.take_along_axis(s, np.maximum(idx, 0), 1), 0.0)
    D = np.maximum(got.sum(1, keepdims=True), 1e-300) if normalize else np.ones((N, 1))
    T = int(routed.sum())
    count = np.bincount(idx[idx >= 0], minlength=E)
    mean = (s / total).sum(0) / max(T, 1)
    f = count / (K * max(T, 1))
    return dict(idx=idx, weights=scale * got / D, count=count, mean=mean, loss=coef * E * float((f * mean).sum()), T=T,
                s=s, total=total, got=got, D=D, f=f, routed=routed)


def plain_backward(r, K, score, normalize, scale, coef, dw, dloss):
    N, E = r["s"].shape
    dw = np.where(r["idx"] >= 0, dw.astype(np.float64), 0.0)
    inner = (dw * r["got"] / r["D"]).sum(1, keepdims=True) if normalize else 0.0
    g = dloss * coef * E * r["f"] / max(r["T"], 1)
    q = r["s"] / r["total"]
    ds = (g - (q * g).sum(1, keepdims=True)) / r["total"]
    mag = (np.abs(g) + (q * np.abs(g)).sum(1, keepdims=True)) / r["total"]
    dk = scale / r["D"] * (dw - inner)
    dk_mag = np.abs(scale / r["D"]) * (np.abs(dw) + np.abs(inner))
    for t in range(N):
        for k in range(K):
            if r["idx"][t, k] >= 0:
                ds[t, r["idx"][t, k]] += dk[t, k]
                mag[t, r["idx"][t, k]] += dk_mag[t, k]
    s = r["s"]
    if score == "softmax":
        dl = s * (ds - (s * ds).sum(1, keepdims=True))
        mag = s * (mag + (s * mag).sum(1, keepdims=True))
    else:
        dl = s * (1 - s) * ds
        mag = s * mag
    dl[~r["routed"]] = 0
    return dl, mag


def draw(N, E, seed, dtype=torch.float32, closed=0.0, empty=0.0, bias=False, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn((N, E), generator=g) * spread
    if closed:
        l[torch.rand((N, E), generator=g) < closed] = float("-inf")
    if empty:
        l[torch.rand(N, generator=g) < empty] = float("-inf")
    b = torch.randn(E, generator=g) * 0.3 if bias else None
    return l.to(dtype), b


def run(l, b, K, cfg, stride=None):
    N, E = l.shape
    desc = binding.LayoutDesc(N, K, E, 1, 1)
    gate = binding.Gate(desc, cfg)
    if stride:
        wide = torch.full((N, stride), float("nan"), dtype=l.dtype, device=DEV)
        wide[:, :E] = l.to(DEV)
        ld = wide[:, :E]
    else:
        ld = l.to(DEV)
    gate.forward(ld, bias=None if b is None else b.to(DEV))
    return gate, ld


def check_forward(gate, r):
    np.testing.assert_array_equal(gate.topk_idx.cpu().numpy(), r["idx"])
    np.testing.assert_array_equal(gate.expert_count.cpu().numpy(), r["count"])
    assert int(gate.routed_tokens) == r["T"]
    w = gate.weights.double().cpu().numpy()
    assert np.all(np.abs(w - r["weights"]) <= 2.0 ** -18 * np.abs(r["weights"]) + 1e-30)
    m = gate.prob_mean.double().cpu().numpy()
    assert np.all(np.abs(m - r["mean"]) <= 2.0 ** -17 * r["mean"] + 1e-30)
    assert abs(float(gate.loss) - r["loss"]) <= 2.0 ** -16 * abs(r["loss"])


CASES = [
    # N, E, K, dtype, score, normalize, bias, closed, empty
    (1, 1, 1, torch.float32, "softmax", True, False, 0, 0),
    (1, 7, 7, torch.float32, "sigmoid", True, False, 0, 0),
    (3, 8, 2, torch.bfloat16, "softmax", False, False, 0, 0),
    (64, 256, 8, torch.float32, "softmax", True, False, 0, 0),
    (257, 384, 8, torch.float32, "softmax", True, False, 0, 0.05),
    (301, 40, 3, torch.bfloat16, "sigmoid", True, True, 0.2, 0.05),
    (130, 33, 32, torch.float32, "softmax", True, True, 0.3, 0.1),
    (95, 64, 6, torch.bfloat16, "softmax", True, True, 0.5, 0.1),
    (77, 100, 1, torch.float32, "sigmoid", False, True, 0, 0),
    (50, 512, 8, torch.float32, "softmax", True, False, 0, 0),
    (60, 1000, 16, torch.bfloat16, "softmax", True, False, 0.1, 0),
    (41, 1024, 32, torch.float32, "sigmoid", True, False, 0, 0),
    (20, 5, 8, torch.float32, "softmax", True, False, 0.4, 0.2),        # more slots than experts
]


@pytest.mark.parametrize("N,E,K,dtype,score,normalize,bias,closed,empty", CASES)
def test_forward_and_backward(N, E, K, dtype, score, normalize, bias, closed, empty):
    l, b = draw(N, E, 100 + N + E, dtype, closed, empty, bias)
    cfg = binding.GateConfig(score, normalize, 2.5, 0.02)
    r = plain(l.float().numpy(), None if b is None else b.numpy(), K, score, normalize, 2.5, 0.02)
    gate, ld = run(l, b, K, cfg)
    assert gate.error() == 0
    check_forward(gate, r)
    g = torch.Generator().manual_seed(7)
    dw, dloss = torch.randn((N, K), generator=g), torch.tensor([1.75])
    dl = torch.full((N, E), 9.0, dtype=dtype, device=DEV)
    gate.backward(ld, dl, dw.to(DEV), dloss.to(DEV))
    assert gate.error() == 0
    want, mag = plain_backward(r, K, score, normalize, 2.5, 0.02, dw.numpy(), 1.75)
    got = dl.double().cpu().numpy()
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    assert np.all(np.abs(got - want) <= step * np.abs(want) + 2.0 ** -16 * mag + 1e-37)


def test_ties_go_to_the_lowest_id():
    l = torch.zeros((5, 70))
    l[0, ::2] = -0.0                     # the two zeros tie
    l[1, 40:] = 1.0
    l[2, [3, 35, 67]] = 2.0
    l[3] = float("-inf")
    l[3, [9, 41]] = -3.4028234663852886e38   # the type's lowest value is a value
    gate, _ = run(l, None, 4, binding.GateConfig("softmax"))
    np.testing.assert_array_equal(gate.topk_idx.cpu().numpy(),
                                  [[0, 1, 2, 3], [40, 41, 42, 43], [3, 35, 67, 0], [9, 41, -1, -1], [0, 1, 2, 3]])
    w = gate.weights.cpu().numpy()
    np.testing.assert_array_equal(w[3], [0.5, 0.5, 0, 0])
    assert gate.error() == 0


def test_lowest_value_as_a_mask_gets_no_weight():
    l = torch.full((2, 16), -3.4028234663852886e38)
    l[0, 5] = 1.0
    gate, _ = run(l, None, 2, binding.GateConfig("softmax"))
    np.testing.assert_array_equal(gate.topk_idx.cpu().numpy(), [[5, 0], [0, 1]])
    np.testing.assert_array_equal(gate.weights.cpu().numpy(), [[1, 0], [0.5, 0.5]])


def test_not_a_number_routes_nowhere_and_is_reported():
    l, _ = draw(40, 24, 3)
    l[4, 7] = float("nan")
    l[9, 0] = float("inf")
    l[11] = float("-inf")
    gate, ld = run(l, None, 3, binding.GateConfig("softmax", True, 1.0, 0.1))
    assert gate.error() == 1
    assert gate.error() == 0
    clean = l.clone()
    clean[[4, 9]] = float("-inf")
    r = plain(clean.numpy(), None, 3, "softmax", True, 1.0, 0.1)
    check_forward(gate, r)
    dl = torch.full((40, 24), 5.0, device=DEV)
    gate.backward(ld, dl, torch.ones((40, 3), device=DEV), torch.ones(1, device=DEV))
    assert torch.all(dl[[4, 9, 11]] == 0) and torch.isfinite(dl).all()


def test_padding_columns_of_a_strided_row_are_not_read():
    l, b = draw(33, 40, 5, torch.bfloat16, 0.1, 0, True)
    cfg = binding.GateConfig("sigmoid", True, 1.0, 0.1)
    gate, ld = run(l, b, 3, cfg, stride=57)
    check_forward(gate, plain(l.float().numpy(), b.numpy(), 3, "sigmoid", True, 1.0, 0.1))
    wide = torch.full((33, 91), 4.0, dtype=torch.bfloat16, device=DEV)
    gate.backward(ld, wide[:, :40], torch.ones((33, 3), device=DEV))
    assert torch.all(wide[:, 40:] == 4.0) and not torch.any(wide[:, :40] == 4.0)
    assert gate.error() == 0


def test_no_tokens_and_no_routed_tokens():
    for N in (0, 37):
        l = torch.full((N, 12), float("-inf"))
        gate, ld = run(l, None, 2, binding.GateConfig(balance_coef=1.0))
        assert int(gate.routed_tokens) == 0 and float(gate.loss) == 0
        assert torch.all(gate.prob_mean == 0) and torch.all(gate.expert_count == 0)
        assert torch.all(gate.topk_idx == -1) and torch.all(gate.weights == 0)
        dl = torch.ones((N, 12), device=DEV)
        gate.backward(ld, dl, torch.ones((N, 2), device=DEV), torch.ones(1, device=DEV))
        assert torch.all(dl == 0) and gate.error() == 0


def test_large_batch_many_ctas_is_deterministic():
    N, E, K = 40000, 96, 4
    l, _ = draw(N, E, 11)
    cfg = binding.GateConfig("softmax", True, 1.0, 0.01)
    gate, ld = run(l, None, K, cfg)
    first = [t.clone() for t in (gate.topk_idx, gate.weights, gate.expert_count, gate.prob_mean, gate.loss)]
    p = torch.softmax(l.double(), 1)
    top = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :K]
    assert torch.equal(gate.topk_idx.cpu(), top)
    assert torch.equal(gate.expert_count.cpu().long(), torch.bincount(top.reshape(-1), minlength=E))
    assert torch.allclose(gate.prob_mean.double().cpu(), p.mean(0), rtol=2.0 ** -17, atol=0)
    for _ in range(3):
        gate.forward(ld)
        for a, b in zip(first, (gate.topk_idx, gate.weights, gate.expert_count, gate.prob_mean, gate.loss)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("score,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_gradient_against_differences(score, normalize):
    """Central differences of the 64-bit loss; the step (1e-5) and curvature leave ~1e-8 of the largest gradient."""
    N, E, K = 9, 20, 3
    l, _ = draw(N, E, 21)
    cfg = binding.GateConfig(score, normalize, 1.5, 0.5)
    gate, ld = run(l, None, K, cfg)
    dw = torch.randn((N, K), generator=torch.Generator().manual_seed(2))
    dl = torch.empty((N, E), device=DEV)
    gate.backward(ld, dl, dw.to(DEV), torch.ones(1, device=DEV))
    base = plain(l.numpy(), None, K, score, normalize, 1.5, 0.5)

    def loss(x):
        if score == "softmax":
            s = np.exp(x - x.max(1, keepdims=True))
            s /= s.sum(1, keepdims=True)
        else:
            s = 1 / (1 + np.exp(-x))
        got = np.take_along_axis(s, base["idx"], 1)
        D = got.sum(1, keepdims=True) if normalize else 1.0
        mean = (s / s.sum(1, keepdims=True)).mean(0)
        return float((dw.numpy() * 1.5 * got / D).sum()) + 0.5 * E * float((base["f"] * mean).sum())

    x = l.double().numpy()
    num = np.zeros_like(x)
    for i in range(N):
        for j in range(E):
            up, dn = x.copy(), x.copy()
            up[i, j] += 1e-5
            dn[i, j] -= 1e-5
            num[i, j] = (loss(up) - loss(dn)) / 2e-5
    got = dl.double().cpu().numpy()
    assert np.abs(got - num).max() <= 1e-5 * np.abs(num).max()


def test_feeds_the_layout_on_another_stream():
    N, E, K = 500, 16, 2
    l, _ = draw(N, E, 31, empty=0.1)
    s = torch.cuda.Stream()
    ld = l.to(DEV)
    desc = binding.LayoutDesc(N, K, E, 4, 8)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        gate = binding.Gate(desc, binding.GateConfig())
        gate.forward(ld)
        lay = binding.Layout(desc, N * K + E * 7)
        lay.build(gate.topk_idx)
    s.synchronize()
    assert torch.equal(lay.expert_count, gate.expert_count)
    assert gate.error() == 0 and lay.error() == 0


def test_refusals():
    desc = binding.LayoutDesc(4, 2, 8, 1, 1)
    gate = binding.Gate(desc, binding.GateConfig())
    ok = torch.zeros((4, 8), device=DEV)
    with pytest.raises(ValueError):
        gate.forward(torch.zeros((4, 9), device=DEV))
    with pytest.raises(ValueError):
        gate.forward(torch.zeros((4, 8), dtype=torch.float16, device=DEV))
    with pytest.raises(ValueError):
        gate.forward(torch.zeros((8, 4), device=DEV).t())
    with pytest.raises(ValueError):
        gate.forward(torch.zeros((4, 8)))
    with pytest.raises(ValueError):
        gate.forward(ok, bias=torch.zeros(7, device=DEV))
    with pytest.raises(ValueError):
        binding.Gate(desc, binding.GateConfig(score="relu")).forward(ok)
    gate.forward(ok)
    with pytest.raises(ValueError):
        gate.backward(ok, torch.zeros((4, 8), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        gate.backward(ok, torch.zeros((4, 8), device=DEV), dweights=torch.zeros((4, 1), device=DEV))


def test_backward_refuses_ids_out_of_range():
    desc = binding.LayoutDesc(4, 2, 8, 1, 1)
    gate = binding.Gate(desc, binding.GateConfig())
    ok = torch.randn((4, 8), device=DEV)
    gate.forward(ok)
    gate.topk_idx[2, 1] = 8
    dl = torch.zeros((4, 8), device=DEV)
    gate.backward(ok, dl, torch.ones((4, 2), device=DEV))
    assert gate.error() == 3 and torch.isfinite(dl).all()
