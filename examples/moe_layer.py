"""A mixture-of-experts layer in 8-bit floating point on the library's calls.

    python examples/moe_layer.py            # one serving pass and one training step on cuda:0

Serving (``MoELayer.serve``): gate -> 8-bit rows -> layout and dispatch -> gate/up
product -> SwiGLU -> down product -> combine.  Rows travel through the dispatch in
8 bits with their scales in the column-major form the product reads.

Training (``MoELayer.step``): the same with bf16 rows dispatched (the weight
gradients quantise them down the columns too), then every gradient: expert
weights, router, and the input's share through the experts.  The weighted sum's
own gradient (a product of rows and a dot product) and the activation's bf16 rows
for the second weight gradient are plain torch here.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from counting_sort_bucketization_gb300 import binding  # noqa: E402

E4M3 = torch.float8_e4m3fn
BLOCK = 128


def quantize_weights(w: torch.Tensor):
    """[E, out, in] to e4m3 with a scale for each 128x128 block; laid out once."""
    E, O, I = w.shape
    ob, ib = -(-O // BLOCK), -(-I // BLOCK)
    v = torch.nn.functional.pad(w.float(), (0, ib * BLOCK - I, 0, ob * BLOCK - O)).view(E, ob, BLOCK, ib, BLOCK)
    sf = v.abs().amax((2, 4)).clamp(min=1e-30) / 448.0
    q = (v / sf[:, :, None, :, None]).reshape(E, ob * BLOCK, ib * BLOCK)[:, :O, :I]
    return q.to(E4M3).contiguous(), sf.contiguous()


def transpose_weights(q: torch.Tensor, sf: torch.Tensor):
    """The operands of the input gradient: a square block keeps its scale when transposed."""
    return q.view(torch.uint8).transpose(1, 2).contiguous().view(E4M3), sf.transpose(1, 2).contiguous()


class MoELayer:
    def __init__(self, hidden, width, num_experts, topk, num_ranks=1, alignment=128, balance_coef=0.01, seed=0,
                 device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s, scale: torch.randn(s, generator=g, device=device) * scale
        self.hidden, self.width, self.E, self.K = hidden, width, num_experts, topk
        self.R, self.A, self.device = num_ranks, alignment, device
        self.router = rand(num_experts, hidden, scale=hidden ** -0.5)
        self.gate_up, self.gate_up_sf = quantize_weights(rand(num_experts, 2 * width, hidden, scale=hidden ** -0.5))
        self.down, self.down_sf = quantize_weights(rand(num_experts, hidden, width, scale=width ** -0.5))
        self.cfg = binding.GateConfig(score="softmax", normalize=True, scale=1.0, balance_coef=balance_coef)

    def _plan(self, N):
        """Buffers of one batch size."""
        desc = binding.LayoutDesc(N, self.K, self.E, self.R, self.A)
        cap = N * self.K + self.E * (self.A - 1)
        cap = -(-cap // BLOCK) * BLOCK
        return desc, cap, binding.Gate(desc, self.cfg, self.device), binding.Layout(desc, cap, self.device)

    def _empty(self, *shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device=self.device)

    def serve(self, x):
        N, H, I = x.shape[0], self.hidden, self.width
        desc, cap, gate, lay = self._plan(N)
        gate.forward(x.float() @ self.router.t())
        lay.build(gate.topk_idx)
        q, sf = self._empty(N, H, dtype=E4M3), self._empty(N, -(-H // BLOCK), dtype=torch.float32)
        binding.quantize_rows(x, q, sf)
        recv, recv_sf = self._empty(cap, H, dtype=E4M3), binding.new_sf_col_major(sf.shape[1], cap, device=self.device)
        lay.permute(q, recv)
        lay.permute_sf_col_major(sf, recv_sf)
        y = self._experts(lay, recv, recv_sf, cap)[-1]
        out = self._empty(N, H)
        lay.combine(y, gate.weights, out)
        self.check(gate, lay)
        return out

    def _experts(self, lay, recv, recv_sf, cap):
        H, I = self.hidden, self.width
        gu = self._empty(cap, 2 * I)
        lay.expert_gemm(recv, recv_sf, self.gate_up, self.gate_up_sf, gu)
        h, h_sf = self._empty(cap, I, dtype=E4M3), binding.new_sf_col_major(-(-I // BLOCK), cap, device=self.device)
        binding.swiglu_quantize(gu, h, h_sf, total_rows=lay.total_rows)
        y = self._empty(cap, H)
        lay.expert_gemm(h, h_sf, self.down, self.down_sf, y)
        return gu, y

    def _rows(self, t, total):
        q, sf = self._empty(*t.shape, dtype=E4M3), binding.new_sf_col_major(-(-t.shape[1] // BLOCK), t.shape[0], device=self.device)
        binding.quantize_rows(t, q, sf, total_rows=total, col_major=True)
        return q, sf

    def _cols(self, lay, t):
        q = self._empty(t.shape[1], -(-t.shape[0] // BLOCK) * BLOCK, dtype=E4M3)
        sf = self._empty(-(-t.shape[0] // BLOCK), t.shape[1], dtype=torch.float32)
        lay.quantize_cols(t, q, sf)
        return q, sf

    def step(self, x, dout):
        """Output, balance loss, and the gradients of out . dout + loss."""
        N, H, I, E, K = x.shape[0], self.hidden, self.width, self.E, self.K
        desc, cap, gate, lay = self._plan(N)
        logits = x.float() @ self.router.t()
        gate.forward(logits)
        lay.build(gate.topk_idx)
        recv = self._empty(cap, H)
        lay.permute(x, recv)
        xq, xsf = self._rows(recv, lay.total_rows)
        gu, y = self._experts(lay, xq, xsf, cap)
        out = self._empty(N, H)
        lay.combine(y, gate.weights, out)

        # the weighted sum: y_row's gradient is its weight times the token's, a weight's the rows' dot product
        slot = lay.dst_slot[: N * K].long()
        routed = slot >= 0
        at = slot.clamp(min=0)
        token = torch.arange(N * K, device=self.device) // K
        dy = torch.zeros((cap, H), dtype=torch.bfloat16, device=self.device)
        dy[at[routed]] = (gate.weights.view(-1, 1) * dout.float()[token])[routed].to(torch.bfloat16)
        dweights = torch.where(routed, (y.float()[at] * dout.float()[token]).sum(1), 0.0).view(N, K)

        down_t, gate_up_t = transpose_weights(self.down, self.down_sf), transpose_weights(self.gate_up, self.gate_up_sf)
        dh = self._empty(cap, I)
        lay.expert_gemm(*self._rows(dy, lay.total_rows), *down_t, dh)
        dgu = self._empty(cap, 2 * I)
        binding.swiglu_backward(gu, dh, dgu, total_rows=lay.total_rows)
        dx_rows = self._empty(cap, H)
        lay.expert_gemm(*self._rows(dgu, lay.total_rows), *gate_up_t, dx_rows)
        dx = self._empty(N, H)
        lay.combine(dx_rows, torch.ones((N, K), device=self.device), dx)

        # from gate_up, not from the 8-bit h: the columns are rounded to 8 bits once
        a, b = gu.float().split(I, 1)
        h_rows = (torch.nn.functional.silu(a) * b).to(torch.bfloat16)
        d_down = torch.empty((E, H, I), device=self.device)
        lay.expert_wgrad(*self._cols(lay, dy), *self._cols(lay, h_rows), d_down)
        d_gate_up = torch.empty((E, 2 * I, H), device=self.device)
        lay.expert_wgrad(*self._cols(lay, dgu), *self._cols(lay, recv), d_gate_up)

        dlogits = torch.empty_like(logits)
        gate.backward(logits, dlogits, dweights, torch.ones(1, device=self.device))
        self.check(gate, lay)
        return dict(out=out, loss=gate.loss, expert_count=gate.expert_count, dx=dx + (dlogits @ self.router).to(dx.dtype),
                    router=dlogits.t() @ x.float(), gate_up=d_gate_up, down=d_down)

    @staticmethod
    def check(gate, lay):
        for name, code in (("gate", gate.error()), ("layout", lay.error())):
            if code:
                raise RuntimeError(f"{name}: {binding.ERROR_NAMES.get(code, code)}")


if __name__ == "__main__":
    layer = MoELayer(hidden=1024, width=512, num_experts=16, topk=4)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((2000, 1024), generator=g, device="cuda").to(torch.bfloat16)
    dout = torch.randn((2000, 1024), generator=g, device="cuda").to(torch.bfloat16)
    served = layer.serve(x)
    got = layer.step(x, dout)
    print("one token:", tuple(layer.serve(x[:1]).shape), " serving and training outputs differ by",
          float((served.float() - got["out"].float()).norm() / served.float().norm()))
    print("balance loss", float(got["loss"]), " tokens an expert", got["expert_count"].tolist())
    print("gradient norms", {k: round(float(got[k].float().norm()), 4) for k in ("dx", "router", "gate_up", "down")})
