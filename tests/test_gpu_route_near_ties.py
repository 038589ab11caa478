"""Routing where the picks tie exactly and a key behind them is the same in 32 bits but a larger number.

All scores and biases are equal but for one or two experts with high ids, whose score is 2^-26 larger: a quarter of
a unit of the key's last place, so 32 bits show ties alone, which go to the lower ids.  As numbers those experts come first
(sigmoid(2^-24) = 1/2 + 2^-26 to 2^-74; keys of 1/2 + 1/4, known to 2^-46).
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


@pytest.mark.parametrize("N", [1, 5000])
@pytest.mark.parametrize("E,K,G,kept", [(8, 2, 1, 1), (24, 4, 1, 1), (32, 8, 1, 1), (40, 6, 1, 1), (96, 8, 1, 1), (384, 8, 1, 1), (1024, 16, 1, 1),
                                       (96, 4, 3, 2), (64, 6, 32, 20), (320, 8, 5, 2), (60, 4, 4, 2)])
def test_a_larger_number_behind_ties(E, K, G, kept, N):
    l = torch.zeros((N, E), device=DEV)
    b = torch.full((E,), 0.25, device=DEV)
    b[0] = 0.125                                           # biases that differ
    per = E // G
    first = E - 1 - torch.arange(N, device=DEV) % 2        # the last expert, or the one before it
    l.scatter_(1, first[:, None], 2.0 ** -24)
    second = E - 1 - per * (torch.arange(N, device=DEV) % 3 == 2).long() if G > 1 else first
    l.scatter_(1, second[:, None], 2.0 ** -24)
    key = torch.sigmoid(l.double()) + b.double()
    gate = binding.Gate(binding.LayoutDesc(N, K, E, 1, 1),
                        binding.GateConfig("sigmoid", bias_on="score", num_groups=G, topk_groups=kept, group_sum=1)).forward(l, bias=b)
    if kept < G:
        best = key.view(N, G, per).amax(2)
        top = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :kept]
        keep = torch.zeros((N, G), dtype=torch.bool, device=DEV).scatter_(1, top, True)
        key = torch.where(keep.repeat_interleave(per, 1), key, -9.0)
    want = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :K]
    assert torch.all(want[:, 0] >= E - 1 - per)
    assert torch.equal(gate.topk_idx, want) and gate.error() == 0
