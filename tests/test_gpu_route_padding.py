"""Routing of padded batches: what a row whose K-th key is a mask leaves behind in its warp is gone after the next one.

A batch of which 3 % of the rows have five experts beside masks of -1e9, the rest closed.  The lists' bound falls to the
masks there and has to rise with the next ordinary row: a row for each halving of 1e9, most of the batch, costs 8 to 12 %.
Ids against 64-bit torch; time, the least of several calls, against the same batch with those masks closed (measured
1 to 2 % apart; 6 % allowed).
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


@pytest.mark.parametrize("E", [32, 64, 128])
def test_masks_leave_no_bound_behind(E):
    N, K = 1 << 19, 8
    g = torch.Generator(device=DEV).manual_seed(1)
    l = torch.randn((N, E), generator=g, device=DEV) * 1.5
    some = (torch.rand((N, 1), generator=g, device=DEV) < 0.03) & (torch.arange(E, device=DEV) >= 5)
    gate = binding.Gate(binding.LayoutDesc(N, K, E, 1, 1), binding.GateConfig("sigmoid", True, 2.5, 0.02, bias_on="score"))
    rows = [torch.where(some, float("-inf"), l)]
    rows.append(torch.where(some & (torch.arange(E, device=DEV) < 5 + 24), -1e9, rows[0]))
    times = [[], []]
    for _ in range(15):
        for l, t in zip(rows, times):
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            gate.forward(l)
            end.record()
            torch.cuda.synchronize()
            t.append(start.elapsed_time(end))
    top = torch.sort(rows[1].double(), dim=1, descending=True, stable=True)
    assert torch.equal(gate.topk_idx, torch.where(top.values[:, :K] > float("-inf"), top.indices[:, :K], -1))
    assert gate.error() == 0
    assert min(times[1]) < 1.06 * min(times[0])
