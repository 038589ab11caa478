"""The example layer's second weight gradient takes the activation rounded to 8 bits once, down the columns."""
from __future__ import annotations

import os
import sys

import pytest
import torch

from counting_sort_bucketization_gb300 import binding, build

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.load_library()


def test_the_activation_reaches_the_columns_in_bf16(monkeypatch):
    """Rows given to quantize_cols for the down projection: silu(gate) * up within one bf16 rounding (2^-9 relative, doubled
    for the fp32 steps before it), not values of 8 bits."""
    from moe_layer import MoELayer

    seen, columns = {}, []
    swiglu, cols = binding.swiglu_quantize, binding.Layout.quantize_cols
    monkeypatch.setattr(binding, "swiglu_quantize", lambda gu, *a, **k: (seen.update(gu=gu), swiglu(gu, *a, **k))[1])
    monkeypatch.setattr(binding.Layout, "quantize_cols",
                        lambda self, x, q, sf, **k: (columns.append((x, int(self.total_rows))), cols(self, x, q, sf, **k))[1])
    layer = MoELayer(256, 128, 8, 2, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    x, dout = (torch.randn((500, 256), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    layer.step(x, dout)
    given = [(t, n) for t, n in columns if t.shape[1] == layer.width]
    assert len(given) == 1
    rows, total = given[0]
    a, b = seen["gu"][:total].double().split(layer.width, 1)
    want = a * torch.sigmoid(a) * b
    assert torch.all((rows[:total].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-30)
