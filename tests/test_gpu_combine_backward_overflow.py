"""Gradient of the combine on a layout that needed more rows than there are: nothing of the rows is written, its gaps
neither, also where dy lies over the expert outputs."""
from __future__ import annotations

import pytest
import torch

from counting_sort_bucketization_gb300 import binding, build

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.load_library()


@pytest.mark.parametrize("N,H", [(30, 64), (30, 2048), (2000, 256)])
def test_gaps_stay(N, H):
    K, E, A = 2, 4, 16
    idx = torch.randint(0, E, (N, K), generator=torch.Generator(device=DEV).manual_seed(N), device=DEV)
    need = int(binding.Layout(binding.LayoutDesc(N, K, E, 1, A), N * K + E * A).build(idx).expert_offset[E])
    for cap, fits in ((need - 1, False), (A, False), (need, True)):
        lay = binding.Layout(binding.LayoutDesc(N, K, E, 1, A), cap).build(idx)
        assert lay.error() == (0 if fits else 4)
        y = torch.full((cap, H), 7.0, dtype=BF16, device=DEV)
        dw = torch.full((N, K), 9.0, device=DEV)
        lay.combine_backward(torch.ones((N, H), dtype=BF16, device=DEV), torch.ones((N, K), device=DEV), y, y, dw)
        assert lay.error() == 0
        if fits:
            gaps = torch.ones(cap, dtype=torch.bool, device=DEV)
            gaps[lay.dst_slot[:N * K].long()] = False
            assert int(gaps.sum()) > 0 and not y[gaps].any() and torch.all(y[~gaps] == 1.0) and torch.all(dw == 7.0 * H)
        else:
            assert torch.all(y == 7.0) and torch.all(dw == 0.0)
