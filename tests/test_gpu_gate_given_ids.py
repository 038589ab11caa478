"""The gate's gradient for ids that the caller chose, among them experts that a mask closes: they score nothing, so their
weight has no gradient, and nothing becomes NaN."""
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_ids_of_closed_experts(score, normalize, dtype):
    E, K = 12, 2
    l = torch.randn((4, E), generator=torch.Generator().manual_seed(1)).to(dtype)
    l[0, [3, 7]] = float("-inf")         # both picks closed
    l[1, 3] = float("-inf")              # one of them
    l[2] = float("-inf")                 # the whole row
    ids = torch.tensor([[3, 7]] * 4)
    dw = torch.tensor([[1.0, -2.0]] * 4)
    desc = binding.LayoutDesc(4, K, E, 1, 1)
    ws = binding.new_gate_workspace(desc)
    count = torch.bincount(ids.reshape(-1), minlength=E).to(torch.int32).to(DEV)
    routed = torch.tensor([4], dtype=torch.int32, device=DEV)
    dl = torch.full((4, E), 9.0, dtype=dtype, device=DEV)
    binding.gate_backward(desc, binding.GateConfig(score, normalize, 1.5, 0.2), l.to(DEV), ids.to(DEV), count, routed, dl, ws,
                          dweights=dw.to(DEV), dloss=torch.ones(1, device=DEV))
    assert binding.get_error(ws) == 0
    assert torch.isfinite(dl).all()
    assert torch.all(dl[0, [3, 7]] == 0) and dl[1, 3] == 0 and torch.all(dl[2] == 0)
    leaf = l.double().requires_grad_()
    s = torch.softmax(leaf[[0, 1, 3]], 1) if score == "softmax" else torch.sigmoid(leaf[[0, 1, 3]])
    p = s.gather(1, ids[:3])
    if normalize:
        p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    q = s / s.sum(1, keepdim=True)
    f = count.cpu().double() / (K * 4)
    (1.5 * (p * dw[:3]).sum() + 0.2 * E * (f * q.sum(0) / 4).sum()).backward()
    want = torch.nan_to_num(leaf.grad)   # differentiating the reference at -inf is 0 * inf there
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -18
    assert torch.all((dl.cpu().double() - want).abs()[[0, 1, 3]] <= step * want.abs()[[0, 1, 3]] + 2.0 ** -18)
