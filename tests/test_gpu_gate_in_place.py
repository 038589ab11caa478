"""The gate's gradient written over the logits it is computed from."""
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


@pytest.mark.parametrize("score,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("N,E,K,dtype,stride", [(30000, 64, 8, torch.float32, 64), (20001, 40, 32, torch.bfloat16, 57),
                                                (5000, 384, 8, torch.float32, 384), (777, 1000, 4, torch.bfloat16, 1001)])
def test_in_place_gives_what_a_buffer_of_its_own_gets(N, E, K, dtype, stride, score, normalize):
    g = torch.Generator(device=DEV).manual_seed(E + N)
    held = torch.randn((N, stride), generator=g, device=DEV).to(dtype)
    held[torch.rand(N, generator=g, device=DEV) < 0.02, :E] = float("-inf")
    held[5, :E] = -90.0
    logits = held[:, :E]
    before = held.clone()
    gate = binding.Gate(binding.LayoutDesc(N, K, E, 1, 1), binding.GateConfig(score, normalize, 1.5, 0.1))
    gate.forward(logits)
    dw, one = torch.randn((N, K), generator=g, device=DEV), torch.ones(1, device=DEV)
    want = torch.empty((N, E), dtype=dtype, device=DEV)
    gate.backward(logits, want, dw, one)
    gate.backward(logits, logits, dw, one)
    assert gate.error() == 0
    assert torch.equal(logits, want)
    assert torch.equal(held[:, E:], before[:, E:])


def test_side_by_side_in_one_buffer():
    both = torch.randn((999, 96), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    gate = binding.Gate(binding.LayoutDesc(999, 4, 48, 1, 1), binding.GateConfig("sigmoid", False))
    logits = both[:, :48].clone()
    gate.forward(both[:, :48])
    dw, want = torch.ones((999, 4), device=DEV), torch.empty((999, 48), device=DEV)
    gate.backward(logits, want, dw)
    gate.backward(both[:, :48], both[:, 48:], dw)
    assert torch.equal(both[:, 48:], want) and torch.equal(both[:, :48], logits)


def test_rows_that_touch_are_refused():
    wide = torch.zeros((8, 20), device=DEV)
    gate = binding.Gate(binding.LayoutDesc(8, 2, 12, 1, 1), binding.GateConfig())
    gate.forward(wide[:, :12])
    with pytest.raises(binding.LayoutError) as e:
        gate.backward(wide[:, :12], wide[:, 8:])
    assert e.value.status == 1
