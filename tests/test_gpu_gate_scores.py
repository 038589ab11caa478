"""Gate scores far from zero.

The plain side works with logarithms in 64 bits, so no score underflows there.

Tolerances.  Logits are multiples of 2^-6 below 2^17 in magnitude, so differences of two are exact in fp32.  An
exponential errs by 2^-22 relative, a reciprocal or approximate quotient by 2^-22, every other operation by 2^-24.  A
score is an exponential, a sum of two, a reciprocal and a product: below 2^-21 whatever its logit.  A sum over at most 64
experts adds 7 roundings, and a weight or probability divides two of those: below 2^-19.
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


def log_sum(x):
    m = x.max(1, keepdims=True)
    return m + np.log(np.exp(x - m).sum(1, keepdims=True))


def plain(l32, bias, K, score, normalize, scale, coef):
    """Every row routes.  log s, log(1 - s), log q and the picks' shares from logarithms."""
    N, E = l32.shape
    key = l32 if bias is None else (l32 + bias).astype(np.float32)
    idx = np.argsort(-key, axis=1, kind="stable")[:, :K]
    l = l32.astype(np.float64)
    if score == "softmax":
        ls = l - log_sum(l)
        rest = np.zeros_like(ls)
    else:
        soft = np.log1p(np.exp(-np.abs(l)))
        ls, rest = np.minimum(l, 0) - soft, np.minimum(-l, 0) - soft
    q = np.exp(ls - log_sum(ls))
    pick = np.take_along_axis(ls, idx, 1)
    share = np.exp(pick - log_sum(pick)) if normalize else np.exp(pick)
    count = np.bincount(idx.ravel(), minlength=E)
    f = count / (K * N)
    mean = q.mean(0)
    return dict(idx=idx, weights=scale * share, share=share, q=q, rest=np.exp(rest), count=count, f=f, mean=mean,
                loss=coef * E * float(f @ mean))


def check(l, bias, K, score, normalize, weight_tol=2.0 ** -19):
    N, E = l.shape
    cfg = binding.GateConfig(score, normalize, 2.5, 0.5)
    r = plain(l, bias, K, score, normalize, 2.5, 0.5)
    gate = binding.Gate(binding.LayoutDesc(N, K, E, 1, 1), cfg)
    ld = torch.from_numpy(l).to(DEV)
    gate.forward(ld, bias=None if bias is None else torch.from_numpy(bias).to(DEV))
    assert gate.error() == 0
    np.testing.assert_array_equal(gate.topk_idx.cpu().numpy(), r["idx"])
    w = gate.weights.double().cpu().numpy()
    # a score below the smallest normal number may come out as zero
    assert np.all(np.abs(w - r["weights"]) <= weight_tol * r["weights"] + 2.5 * 2.0 ** -126)
    if normalize:
        assert np.all(np.abs(w.sum(1) - 2.5) <= 2.5 * 2.0 ** -19)
    mean = gate.prob_mean.double().cpu().numpy()
    assert np.all(np.abs(mean - r["mean"]) <= 2.0 ** -18 * r["mean"] + 2.0 ** -126)
    assert abs(mean.sum() - 1) <= 2.0 ** -18
    assert abs(float(gate.loss) - r["loss"]) <= 2.0 ** -17 * r["loss"]


@pytest.mark.parametrize("normalize", [True, False])
def test_sigmoid_scores_of_any_magnitude(normalize):
    """Unnormalised weights are the scores: as exact at -60 as at 0."""
    rng = np.random.default_rng(3)
    centre = np.linspace(-60, 4, 200)[:, None]
    l = (np.floor((centre + rng.uniform(-3, 3, (200, 32))) * 64) / 64).astype(np.float32)
    check(l, None, 8, "sigmoid", normalize, 2.0 ** -19 if normalize else 2.0 ** -21)


def test_softmax_scores_of_any_magnitude():
    l = grid(np.random.default_rng(4), 200, 32, lo=-70, hi=0)
    l[:, 7] = 0
    check(l, None, 32, "softmax", False)
