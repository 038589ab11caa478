"""The example block (examples/moe_layer.py: residual, norm, routing by groups, experts and back) against plain
autograd, and a run of its calls captured and replayed.

Bounds as in test_gpu_moe_layer.py: two 8-bit products in a row 8 % of the norm, gradients 12 %.  The norm's weight and
the input's gradient pass through the same products: 12 %.  The choice of experts is not continuous: the plain block
takes the one made on the rounded norm, as the block does.  The balance loss sees the probabilities of rounded rows:
2^-7 (two roundings to bf16 on the way to the logits).
"""
from __future__ import annotations

import os
import sys

import pytest
import torch

from counting_sort_bucketization_gb300 import binding, build

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.load_library()


def off(a, b):
    a, b = a.detach().float(), b.detach().float()
    return float((a - b).norm() / b.norm())


def dequantize(q, sf):
    w = q.float()
    return w * sf.repeat_interleave(128, 1)[:, : w.shape[1]].repeat_interleave(128, 2)[:, :, : w.shape[2]]


def plain(block, x, residual, dout, dresidual):
    """The block in 32 bits by autograd, with the quantised weights' values and the choice made on the rounded norm."""
    layer = block.layer
    x = x.float().requires_grad_()
    weight = block.weight.float().requires_grad_()
    router = layer.router.clone().requires_grad_()
    gate_up = dequantize(layer.gate_up, layer.gate_up_sf).requires_grad_()
    down = dequantize(layer.down, layer.down_sf).requires_grad_()
    z = x + residual.float()
    zr = z.detach().to(BF16).float()
    y = z * torch.rsqrt(z.square().mean(1, keepdim=True) + block.eps) * weight
    yr = (zr * torch.rsqrt(zr.square().mean(1, keepdim=True) + block.eps) * weight.detach()).to(BF16).float()
    gate = binding.Gate(binding.LayoutDesc(x.shape[0], layer.K, layer.E, 1, 1), layer.cfg)
    top = gate.forward(yr @ layer.router.t(), bias=layer.bias).topk_idx
    s = torch.sigmoid(y @ router.t())
    w = s.gather(1, top)
    w = layer.cfg.scale * w / w.sum(1, keepdim=True)
    out = torch.zeros_like(x)
    for e in range(layer.E):
        t, k = torch.nonzero(top == e, as_tuple=True)
        a, b = (y[t] @ gate_up[e].t()).split(layer.width, 1)
        out = out.index_add(0, t, w[t, k].unsqueeze(1) * ((torch.nn.functional.silu(a) * b) @ down[e].t()))
    f = torch.bincount(top.reshape(-1), minlength=layer.E).float() / top.numel()
    loss = layer.cfg.balance_coef * layer.E * (f * (s / s.sum(1, keepdim=True)).mean(0)).sum()
    ((out * dout.float()).sum() + (z * dresidual.float()).sum() + loss).backward()
    return dict(out=out, loss=loss, dx=x.grad, router=router.grad, gate_up=gate_up.grad, down=down.grad, weight=weight.grad)


@pytest.mark.parametrize("N,H,I,E,K,G,kept", [(700, 256, 128, 16, 2, 4, 2), (300, 400, 208, 12, 3, 3, 2)])
def test_block_against_autograd(N, H, I, E, K, G, kept):
    from moe_layer import MoEBlock

    block = MoEBlock(H, I, E, K, G, kept, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    block.weight = (torch.randn(H, generator=g, device="cuda") * 0.2 + 1).to(BF16)
    block.layer.bias = torch.randn(E, generator=g, device="cuda") * 0.05
    x, residual, dout, dres = (torch.randn((N, H), generator=g, device="cuda").to(BF16) for _ in range(4))
    want = plain(block, x, residual, dout, dres)
    bias = block.layer.bias.clone()
    got = block.step(x, residual, dout, dres)
    assert off(got["out"], want["out"]) < 0.08
    assert abs(float(got["loss"]) - float(want["loss"].detach())) < 2.0 ** -7 * float(want["loss"].detach())
    assert int(got["expert_count"].sum()) == N * K
    for k in ("dx", "router", "gate_up", "down", "weight"):
        assert off(got[k], want[k]) < 0.12, k
    count = got["expert_count"].float()
    assert torch.equal(block.layer.bias, bias + block.bias_rate * torch.sign(count.mean() - count))
    block.layer.bias = bias
    stream = residual.clone()
    served = block.serve(x, stream)
    assert torch.equal(stream, got["residual"])
    assert off(served, want["out"]) < 0.08


def test_single_tokens_agree_with_the_batch():
    from moe_layer import MoEBlock

    block = MoEBlock(256, 128, 16, 2, 4, 2, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    x, residual = (torch.randn((6, 256), generator=g, device="cuda").to(BF16) for _ in range(2))
    batch = block.serve(x, residual.clone())
    for t in range(6):
        one = block.serve(x[t:t + 1], residual[t:t + 1].clone())
        assert off(one[0], batch[t]) < 2.0 ** -7


def test_the_run_captured_and_replayed():
    """norm -> routing -> layout -> dispatch -> combine -> its gradient -> gate's and norm's gradients as one graph,
    replayed on other inputs: bit for bit what the calls give one by one."""
    N, H, E, K, A = 200, 512, 32, 4, 16
    g = torch.Generator(device="cuda").manual_seed(7)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")
    router, bias, weight = rand(E, H) * H ** -0.5, rand(E) * 0.05, (rand(H) * 0.1 + 1).to(BF16)
    desc = binding.LayoutDesc(N, K, E, 1, A)
    cap = N * K + E * (A - 1)
    cfg = binding.GateConfig("sigmoid", True, 2.5, 0.01, bias_on="score", num_groups=8, topk_groups=3, group_sum=2)
    ws = binding.new_norm_workspace(H)

    def buffers():
        b16 = lambda *s: torch.zeros(s, dtype=BF16, device="cuda")
        return dict(gate=binding.Gate(desc, cfg), lay=binding.Layout(desc, cap), y=b16(N, H), z=b16(N, H), rstd=torch.zeros(N, device="cuda"),
                    q=torch.zeros((N, H), dtype=torch.float8_e4m3fn, device="cuda"), sf=torch.zeros((N, H // 128), device="cuda"),
                    recv=b16(cap, H), recv8=torch.zeros((cap, H), dtype=torch.float8_e4m3fn, device="cuda"),
                    recv_sf=binding.new_sf_col_major(H // 128, cap).zero_(), out=b16(N, H), dy=b16(cap, H), dw=torch.zeros((N, K), device="cuda"),
                    logits=torch.zeros((N, E), device="cuda"), dlogits=torch.zeros((N, E), device="cuda"), dx=b16(N, H), dz=b16(N, H),
                    dweight=torch.zeros(H, device="cuda"))

    def run(b, x, residual, dout):
        binding.rms_norm(x, weight, y=b["y"], q=b["q"], sf=b["sf"], residual=residual, residual_out=b["z"], rstd=b["rstd"])
        torch.mm(b["y"].float(), router.t(), out=b["logits"])
        b["gate"].forward(b["logits"], bias=bias)
        lay = b["lay"].build(b["gate"].topk_idx)
        lay.permute(b["y"], b["recv"])
        lay.permute(b["q"], b["recv8"])
        lay.permute_sf_col_major(b["sf"], b["recv_sf"])
        lay.combine(b["recv"], b["gate"].weights, b["out"])
        lay.combine_backward(dout, b["gate"].weights, b["dy"], b["recv"], b["dw"])
        lay.combine(b["dy"], torch.ones_like(b["dw"]), b["dx"])
        b["gate"].backward(b["logits"], b["dlogits"], b["dw"], one)
        binding.rms_norm_backward(b["dx"], b["z"], b["rstd"], weight, b["dz"], dresidual=dout, dweight=b["dweight"], workspace=ws)

    one = torch.ones(1, device="cuda")
    x, residual, dout = (rand(N, H).to(BF16) for _ in range(3))
    kept = buffers()
    run(kept, x, residual, dout)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(kept, x, residual, dout)
    for t in (x, residual, dout):
        t.copy_(rand(N, H).to(BF16))
    graph.replay()
    fresh = buffers()
    run(fresh, x, residual, dout)
    torch.cuda.synchronize()
    assert kept["gate"].error() == kept["lay"].error() == fresh["gate"].error() == fresh["lay"].error() == 0
    rows = int(fresh["lay"].total_rows)
    for k in fresh:
        if k == "gate":
            for a in ("topk_idx", "weights", "expert_count", "prob_mean", "loss"):
                assert torch.equal(getattr(kept[k], a), getattr(fresh[k], a)), a
        elif k != "lay":
            a, b = kept[k], fresh[k]
            if a.shape[0] == cap:        # rows past the last segment hold an earlier batch's
                a, b = a[:rows], b[:rows]
            if k == "recv_sf":
                a, b = a[:, :rows], b[:, :rows]
            a, b = (t.view(torch.uint8) if t.element_size() == 1 else t for t in (a, b))
            assert torch.equal(a, b), k
