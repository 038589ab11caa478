"""The example layer (examples/moe_layer.py): every operator in the order a user runs it, against plain autograd.

An e4m3 value errs by at most 2^-4 of itself, in the mean over a block by about 2.6 % (a uniform error over steps of
2^-3); a product of two quantised operands of random signs by 3.7 % of its norm, and two products in a row with the
activation between them by 6.5 %.  Gradients pass up to four: 9 %.  Bounds: 8 % and 12 % of the norm.
"""
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


def dequantize(q, sf):
    w = q.float()
    return w * sf.repeat_interleave(128, 1)[:, : w.shape[1]].repeat_interleave(128, 2)[:, :, : w.shape[2]]


def plain(layer, x, dout):
    """The layer in 32 bits by autograd, with the quantised weights' values."""
    x = x.float().requires_grad_()
    router = layer.router.clone().requires_grad_()
    gate_up = dequantize(layer.gate_up, layer.gate_up_sf).requires_grad_()
    down = dequantize(layer.down, layer.down_sf).requires_grad_()
    p = torch.softmax(x @ router.t(), 1)
    top = torch.sort(x.detach() @ router.t().detach(), dim=1, descending=True, stable=True).indices[:, : layer.K]
    w = p.gather(1, top)
    w = w / w.sum(1, keepdim=True)
    out = torch.zeros_like(x)
    for e in range(layer.E):
        t, k = torch.nonzero(top == e, as_tuple=True)
        a, b = (x[t] @ gate_up[e].t()).split(layer.width, 1)
        out = out.index_add(0, t, w[t, k].unsqueeze(1) * ((torch.nn.functional.silu(a) * b) @ down[e].t()))
    f = torch.bincount(top.reshape(-1), minlength=layer.E).float() / top.numel()
    loss = layer.cfg.balance_coef * layer.E * (f * p.mean(0)).sum()
    ((out * dout.float()).sum() + loss).backward()
    return dict(out=out, loss=loss, dx=x.grad, router=router.grad, gate_up=gate_up.grad, down=down.grad)


def off(a, b):
    a, b = a.detach().float(), b.detach().float()
    return float((a - b).norm() / b.norm())


@pytest.mark.parametrize("N,H,I,E,K", [(700, 256, 128, 8, 2), (300, 400, 208, 5, 3)])
def test_layer_against_autograd(N, H, I, E, K):
    from moe_layer import MoELayer

    layer = MoELayer(H, I, E, K, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((N, H), generator=g, device="cuda").to(torch.bfloat16)
    dout = torch.randn((N, H), generator=g, device="cuda").to(torch.bfloat16)
    want = plain(layer, x, dout)
    got = layer.step(x, dout)
    assert off(got["out"], want["out"]) < 0.08
    assert abs(float(got["loss"]) - float(want["loss"].detach())) < 1e-5 * float(want["loss"].detach())
    assert int(got["expert_count"].sum()) == N * K
    for k in ("dx", "router", "gate_up", "down"):
        assert off(got[k], want[k]) < 0.12, k
    assert off(layer.serve(x), want["out"]) < 0.08


def test_single_tokens_agree_with_the_batch():
    from moe_layer import MoELayer

    layer = MoELayer(256, 128, 8, 2, seed=5)
    x = torch.randn((6, 256), generator=torch.Generator(device="cuda").manual_seed(6), device="cuda").to(torch.bfloat16)
    batch = layer.serve(x)
    for t in range(6):
        one = layer.serve(x[t:t + 1])
        # the same products; K may be split over a cluster, so sums may round differently
        assert off(one[0], batch[t]) < 2.0 ** -7
