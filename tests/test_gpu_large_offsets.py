"""Buffers of more than 2^31 elements: the last rows of the norm, of its gradient, of the combine's gradient and of the
routing come from where they lie, and rows that are not named stay as they were."""
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
    yield
    torch.cuda.empty_cache()


def rand(*s, seed=0):
    return torch.randn(s, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(BF16)


def test_norm():
    R, C = 140000, 16384                         # 2.29e9 values
    x, y, dz = (torch.zeros((R, C), dtype=BF16, device=DEV) for _ in range(3))
    x[-3:] = rand(3, C)
    w, rstd, dw = rand(C, seed=1), torch.empty(R, device=DEV), torch.empty(C, device=DEV)
    binding.rms_norm(x, w, y=y, rstd=rstd)
    z = x[-3:].double()
    r = (z.square().mean(1, keepdim=True) + 1e-6).rsqrt()
    want = z * r * w.double()
    assert torch.all((y[-3:].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -16) * want.abs()) and not y[:-3].any()
    y.zero_()
    y[-3:] = rand(3, C, seed=2)                   # now the gradient
    binding.rms_norm_backward(y, x, rstd, w, dz, dweight=dw, workspace=binding.new_norm_workspace(C))
    g, h = y[-3:].double() * w.double(), z * r
    want = r * (g - h * (g * h).mean(1, keepdim=True))
    off = 2.0 ** -16 * (r * (g.abs() + h.abs() * (g * h).abs().mean(1, keepdim=True)))
    assert torch.all((dz[-3:].double() - want).abs() <= off + 2.0 ** -8 * want.abs()) and not dz[:-3].any()
    want = (y[-3:].double() * h).sum(0)
    assert torch.all((dw.double() - want).abs() <= 2.0 ** -16 * (y[-3:].double() * h).abs().sum(0))


def test_combine_gradient():
    H, cap = 8192, 300000                        # 2.46e9 values
    idx = torch.zeros((cap, 1), dtype=torch.int64, device=DEV)
    lay = binding.Layout(binding.LayoutDesc(cap, 1, 2, 1, 1), cap).build(idx)
    dout, y, dy = (torch.zeros((cap, H), dtype=BF16, device=DEV) for _ in range(3))
    dout[-2:], y[-2:] = rand(2, H, seed=3), rand(2, H, seed=4)
    w, dw = torch.full((cap, 1), 0.5, device=DEV), torch.empty((cap, 1), device=DEV)
    lay.combine_backward(dout, w, dy, y, dw)
    assert lay.error() == 0
    assert torch.equal(dy[-2:], (0.5 * dout[-2:].float()).to(BF16)) and not dy[:-2].any()
    prod = dout[-2:].double() * y[-2:].double()
    assert torch.all((dw[-2:, 0].double() - prod.sum(1)).abs() <= 2.0 ** -16 * prod.abs().sum(1)) and not dw[:-2].any()


def test_routing():
    N, E, ld = 70000, 32, 32768                  # rows 32768 apart: 2.29e9 values
    l = torch.zeros((N, ld), dtype=BF16, device=DEV)[:, :E]
    l[-5:] = rand(5, E, seed=5)
    gate = binding.Gate(binding.LayoutDesc(N, 4, E, 1, 1),
                        binding.GateConfig("sigmoid", bias_on="score", num_groups=4, topk_groups=2, group_sum=2)).forward(l)
    for t in range(N - 5, N):
        s = torch.sigmoid(l[t].double()).view(4, 8)
        kept = torch.sort(torch.sort(s, dim=1, descending=True).values[:, :2].sum(1), descending=True, stable=True).indices[:2].tolist()
        order = torch.sort(l[t].float(), descending=True, stable=True).indices.tolist()
        assert gate.topk_idx[t].tolist() == [e for e in order if e // 8 in kept][:4]
    assert torch.all(gate.topk_idx[:-5] == torch.arange(4, device=DEV)) and gate.error() == 0
