"""Gate scores far from zero: rows whose scores are all tiny, exponents of large magnitude, saturated sigmoids.

The plain side works with logarithms in 64 bits, so no score underflows there.

Tolerances.  Logits are multiples of 2^-6 below 2^17 in magnitude, so differences of two are exact in fp32.  An
exponential errs by 2^-22 relative, a reciprocal or approximate quotient by 2^-22, every other operation by 2^-24.  A
score is an exponential, a sum of two, a reciprocal and a product: below 2^-21 whatever its logit.  A sum over at most 64
experts adds 7 roundings, and a weight or probability divides two of those: below 2^-19.  A gradient is a sum of
products of five such factors: 2^-17 of the sum of its terms' magnitudes.
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


def grid(rng, *shape, lo, hi):
    """Multiples of 2^-6 in [lo, hi)."""
    return (np.floor(rng.uniform(lo, hi, shape) * 64) / 64).astype(np.float32)


def shares(x):
    """exp(x) / sum(exp(x)) of a row."""
    e = np.exp(x - x.max(1, keepdims=True))
    return e / e.sum(1, keepdims=True)


def plain(l32, bias, K, score, normalize, scale, coef):
    """Every row routes.  log s and log(1 - s); q and the picks' shares from them."""
    N, E = l32.shape
    key = l32 if bias is None else (l32 + bias).astype(np.float32)
    idx = np.argsort(-key, axis=1, kind="stable")[:, :K]
    l = l32.astype(np.float64)
    if score == "softmax":
        ls = l - l.max(1, keepdims=True)
        ls -= np.log(np.exp(ls).sum(1, keepdims=True))
        rest = np.zeros_like(ls)
    else:
        soft = np.log1p(np.exp(-np.abs(l)))
        ls, rest = np.minimum(l, 0) - soft, np.minimum(-l, 0) - soft
    q = shares(ls)
    pick = np.take_along_axis(ls, idx, 1)
    share = shares(pick) if normalize else np.exp(pick)
    count = np.bincount(idx.ravel(), minlength=E)
    f = count / (K * N)
    mean = q.mean(0)
    return dict(idx=idx, weights=scale * share, share=share, q=q, rest=np.exp(rest), count=count, f=f, mean=mean,
                loss=coef * E * float(f @ mean))


def plain_backward(r, score, normalize, scale, coef, dw):
    N, E = r["q"].shape
    g = (coef * E * r["f"] / N)[None]
    A = (r["q"] * g).sum(1, keepdims=True)
    dl, mag = r["q"] * r["rest"] * (g - A), r["q"] * r["rest"] * (np.abs(g) + np.abs(A))
    inner = (r["share"] * dw).sum(1, keepdims=True) if normalize else 0.0
    dk = scale * r["share"] * (dw - inner)
    dk_mag = scale * r["share"] * (np.abs(dw) + np.abs(inner))
    rest = np.take_along_axis(r["rest"], r["idx"], 1)
    for t in range(N):
        for k, e in enumerate(r["idx"][t]):
            dl[t, e] += dk[t, k] * rest[t, k]
            mag[t, e] += dk_mag[t, k] * rest[t, k]
    if score == "softmax" and not normalize:
        dl -= r["q"] * dk.sum(1, keepdims=True)
        mag += r["q"] * dk_mag.sum(1, keepdims=True)
    return dl, mag


def check_forward(l, bias, K, score, normalize, weight_tol=2.0 ** -19):
    N, E = l.shape
    cfg = binding.GateConfig(score, normalize, 2.5, 0.5)
    r = plain(l, bias, K, score, normalize, 2.5, 0.5)
    gate = binding.Gate(binding.LayoutDesc(N, K, E, 1, 1), cfg)
    ld = torch.from_numpy(l).to(DEV)
    gate.forward(ld, bias=None if bias is None else torch.from_numpy(bias).to(DEV))
    assert gate.error() == 0
    np.testing.assert_array_equal(gate.topk_idx.cpu().numpy(), r["idx"])
    w = gate.weights.double().cpu().numpy()
    # what is below the smallest normal number may come out as zero
    assert np.all(np.abs(w - r["weights"]) <= weight_tol * r["weights"] + 2.5 * 2.0 ** -126)
    if normalize:
        assert np.all(np.abs(w.sum(1) - 2.5) <= 2.5 * 2.0 ** -19)
    mean = gate.prob_mean.double().cpu().numpy()
    assert np.all(np.abs(mean - r["mean"]) <= 2.0 ** -18 * r["mean"] + 2.0 ** -126)
    assert abs(mean.sum() - 1) <= 2.0 ** -18
    assert abs(float(gate.loss) - r["loss"]) <= 2.0 ** -17 * r["loss"] + 0.5 * E * 2.0 ** -126
    return gate, ld, r


def check(l, bias, K, score, normalize):
    gate, ld, r = check_forward(l, bias, K, score, normalize)
    N, E = l.shape
    dw = np.random.default_rng(5).standard_normal((N, K)).astype(np.float32)
    dl = torch.full((N, E), 9.0, device=DEV)
    gate.backward(ld, dl, torch.from_numpy(dw).to(DEV), torch.ones(1, device=DEV))
    assert gate.error() == 0
    want, mag = plain_backward(r, score, normalize, 2.5, 0.5, dw.astype(np.float64))
    err = np.abs(dl.double().cpu().numpy() - want)
    assert np.all(err <= 2.0 ** -17 * mag + 2.0 ** -120)


@pytest.mark.parametrize("E,K", [(16, 4), (40, 3), (64, 32)])
@pytest.mark.parametrize("top", [-40.0, -66.0, -72.0, -90.0, -110.0, -1000.0, -100000.0])
def test_sigmoid_rows_whose_scores_are_all_tiny(top, E, K):
    """The weights sum to the scale and the probabilities to one however small the scores are."""
    check(grid(np.random.default_rng(int(-top) + E), 13, E, lo=top - 4, hi=top), None, K, "sigmoid", True)


def test_rows_at_the_lowest_value():
    l = np.full((2, 8), np.finfo(np.float32).min, np.float32)
    l[1, 3] = -1.0
    check(l[:1], None, 4, "sigmoid", True)
    check(l[1:], None, 1, "sigmoid", True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("below", [20.0, 60.0, 85.0, 150.0, 5000.0])
def test_a_bias_that_picks_experts_far_below_the_largest_logit(score, below):
    """The picks' weights are shares of the picks' own scores, all tiny beside the row's largest."""
    rng = np.random.default_rng(int(below))
    l = grid(rng, 9, 48, lo=-3, hi=3)
    l[:, 16:] -= np.float32(below)
    bias = np.zeros(48, np.float32)
    bias[16:] = 2 * below
    check(l, bias, 5, score, True)


@pytest.mark.parametrize("normalize", [True, False])
def test_sigmoid_scores_of_any_magnitude(normalize):
    """Unnormalised weights are the scores: as exact at -80 as at 0."""
    rng = np.random.default_rng(3)
    centre = np.linspace(-78, 4, 200)[:, None]
    l = (np.floor((centre + rng.uniform(-3, 3, (200, 32))) * 64) / 64).astype(np.float32)
    check_forward(l, None, 8, "sigmoid", normalize, 2.0 ** -19 if normalize else 2.0 ** -21)


def test_softmax_scores_of_any_magnitude():
    l = grid(np.random.default_rng(4), 200, 32, lo=-70, hi=0)
    l[:, 7] = 0
    check_forward(l, None, 32, "softmax", False)


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("size", [8.0, 12.0, 16.0, 25.0, 60.0])
def test_sigmoid_gradient_where_scores_are_close_to_one(size, normalize):
    """1 - s is kept to full precision: s itself rounds to one from a logit of 17 on."""
    rng = np.random.default_rng(int(size))
    l = grid(rng, 21, 24, lo=size - 2, hi=size + 2)
    l[rng.random(l.shape) < 0.4] *= -1
    check(l, None, 4, "sigmoid", normalize)
