"""Routing by groups: the gradient by the function and by the object, and groups of saturated scores."""
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


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_the_functions_gradient_is_the_objects(score):
    N, E, K = 3000, 64, 4
    g = torch.Generator(device=DEV).manual_seed(9)
    l, b = torch.randn((N, E), generator=g, device=DEV) * 1.5, torch.randn(E, generator=g, device=DEV) * 0.05
    dw, one = torch.randn((N, K), generator=g, device=DEV), torch.ones(1, device=DEV)
    desc = binding.LayoutDesc(N, K, E, 1, 1)
    cfg = binding.GateConfig(score, True, 2.5, 0.02, bias_on="score", num_groups=8, topk_groups=3, group_sum=2)
    gate = binding.Gate(desc, cfg).forward(l, bias=b)
    out = [torch.empty_like(t) for t in (gate.topk_idx, gate.weights, gate.expert_count, gate.prob_mean, gate.routed_tokens, gate.loss)]
    ws = binding.new_gate_workspace(desc)
    binding.gate_forward(desc, cfg, l, *out, ws, bias=b)
    for loss in (None, one):
        want, got = torch.full_like(l, 7.0), torch.full_like(l, 9.0)
        gate.backward(l, want, dw, loss)
        binding.gate_backward(desc, cfg, l, out[0], out[2], out[4], got, ws, dweights=dw, dloss=loss)
        assert torch.equal(got, want) and want.any() and not torch.any(want == 7.0)
    assert binding.get_error(ws) == 0 and gate.error() == 0


@pytest.mark.parametrize("bias", [None, 0.25])
def test_groups_of_saturated_scores(bias):
    """Scores that differ from 1 by less than 2^-124: by one key the groups go by their logits, by the sum of two they
    tie, and the lower ids stay; the experts of those go by their logits."""
    l = torch.arange(64, dtype=torch.float32, device=DEV).repeat(5000, 1) + 100.0
    b = None if bias is None else torch.full((64,), bias, device=DEV)
    for group_sum, first in ((1, 63), (2, 31)):
        gate = binding.Gate(binding.LayoutDesc(5000, 8, 64, 1, 1),
                            binding.GateConfig("sigmoid", bias_on="score", num_groups=4, topk_groups=2, group_sum=group_sum))
        gate.forward(l, bias=b)
        assert torch.equal(gate.topk_idx, torch.arange(first, first - 8, -1, device=DEV).repeat(5000, 1)) and gate.error() == 0
